// AdamW over a list of tensors with both moments in fp32, and the 2-norm of a
// list of gradients with the factor that clips it (sm_103a).
//
// The 8-bit optimizer keeps some tensors' moments in 32 bits: the embedding
// (its gradients are uneven across rows) and vectors too small to gain from
// 8 bits.  This step is theirs, with the same scalars as the 8-bit one:
//   g' = s g;  m = b1 m + (1-b1) g';  v = b2 v + ((1-b2) g') g';
//   p = p d - step m / (sqrt(v) / c + eps).
// s is read from device memory, so a clipping factor computed on the device
// needs no round trip through the host; where s is not finite nothing is
// written (an overflowed gradient leaves the state as it was).  Whether it is
// the host does not know, so the count of steps, which the bias corrections
// step and c come from, may be held on the device too.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bwd.h"
#include "host_util.h"

namespace {

using bwd::host::aligned16;
using bwd::host::aligned_to;
using bwd::host::check_launch;
using bwd::host::cuda_fail;
using bwd::host::fail;
using bwd::host::StepCount;

constexpr int kF32 = BWD_F32, kBF16 = BWD_BF16, kF16 = BWD_F16;
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 4;                // elements of a CTA: a quad of 4 per thread
constexpr int kMaxTensors = 480;                    // per launch, bounded by kernel parameter space

struct Tensor32 {
  void* p;
  const void* g;
  float* m;
  float* v;
  int64_t n;
  int64_t shift;  // elements that every pointer lies past four of its elements' boundary, or -1 where they differ
};

struct Adam32Args {
  int64_t chunk_start[kMaxTensors + 1];  // prefix sums of per-tensor chunk counts
  Tensor32 t[kMaxTensors];
  const float* grad_scale;  // or null: 1
  const StepCount* count;   // where step_size and inv_bc2s are, or null: here
  int32_t num_tensors;
  float b1, omb1, b2, omb2, eps, step_size, inv_bc2s, decay;
};

constexpr int64_t kMaxChunks = 0x7fffffff;  // CTAs of one launch

static_assert(sizeof(Adam32Args) <= 32764, "kernel parameter space");

template <int kT>
__device__ __forceinline__ float widen(unsigned short h) {
  if (kT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return __half2float(__ushort_as_half(h));
}

template <int kT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if (kT == kF32) return static_cast<const float*>(x)[i];
  return widen<kT>(static_cast<const unsigned short*>(x)[i]);
}

template <int kT>
__device__ __forceinline__ void store1(void* x, int64_t i, float v) {
  if (kT == kF32) static_cast<float*>(x)[i] = v;
  else if (kT == kBF16) static_cast<__nv_bfloat16*>(x)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(x)[i] = __float2half_rn(v);
}

// Four consecutive elements; each byte is read and written once.
template <int kT>
__device__ __forceinline__ void load4(const void* x, int64_t i, float (&o)[4]) {
  if (kT == kF32) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(x) + i));
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  } else {
    const ushort4 a = __ldcs(reinterpret_cast<const ushort4*>(static_cast<const unsigned short*>(x) + i));
    o[0] = widen<kT>(a.x); o[1] = widen<kT>(a.y); o[2] = widen<kT>(a.z); o[3] = widen<kT>(a.w);
  }
}

template <int kT>
__device__ __forceinline__ void store4(void* x, int64_t i, const float (&v)[4]) {
  if (kT == kF32) {
    __stcs(reinterpret_cast<float4*>(static_cast<float*>(x) + i), make_float4(v[0], v[1], v[2], v[3]));
  } else {
    ushort4 h;
    if (kT == kBF16) {
      h.x = __bfloat16_as_ushort(__float2bfloat16_rn(v[0])); h.y = __bfloat16_as_ushort(__float2bfloat16_rn(v[1]));
      h.z = __bfloat16_as_ushort(__float2bfloat16_rn(v[2])); h.w = __bfloat16_as_ushort(__float2bfloat16_rn(v[3]));
    } else {
      h.x = __half_as_ushort(__float2half_rn(v[0])); h.y = __half_as_ushort(__float2half_rn(v[1]));
      h.z = __half_as_ushort(__float2half_rn(v[2])); h.w = __half_as_ushort(__float2half_rn(v[3]));
    }
    __stcs(reinterpret_cast<ushort4*>(static_cast<unsigned short*>(x) + i), h);
  }
}

// The last t with start[t] <= c: uniform reads of the table in parameter
// space (a warp's ballot over 32 entries at a time reads lanes' own entries,
// which that space serves one by one: 292 tensors 1.39 ms against 1.29).
__device__ __forceinline__ int find_tensor(const int64_t* start, int num, int64_t c) {
  int lo = 0, hi = num - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One CTA for each chunk of 1,024 elements.  Bound by DRAM (26 bytes a
// parameter with fp32 parameters and bf16 gradients).  Against CTAs that walk
// the chunks, four to an SM with twice the elements each, 32000 x 4096 bf16
// parameters take 408 us instead of 431 (7.1 TB/s), and all of a 355M set
// 1.29 ms instead of 1.43; prefetches of the next chunk into L2 made those
// slower still (497 us).
template <int kG, int kP>
__global__ void __launch_bounds__(kThreads)
adam32_kernel(const __grid_constant__ Adam32Args a) {
  const int ti = find_tensor(a.chunk_start, a.num_tensors, blockIdx.x);
  const Tensor32& T = a.t[ti];
  // Quads lie on boundaries in memory: of a tensor that starts between two,
  // the first quad holds fewer elements.  Where the four arrays start
  // differently, a thread's elements are a CTA apart, so that a warp's still
  // follow one another.
  const int64_t base = (blockIdx.x - a.chunk_start[ti]) * kChunk;
  const bool together = T.shift >= 0;
  const int64_t i = together ? base - T.shift + 4 * threadIdx.x : base + threadIdx.x;
  const int step = together ? 1 : kThreads;
  const bool vec = together && i >= 0 && i + 4 <= T.n;
  float p[4], g[4], m[4], v[4];
  if (vec) {
    load4<kP>(T.p, i, p); load4<kG>(T.g, i, g);
    load4<kF32>(T.m, i, m); load4<kF32>(T.v, i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t e = i + j * step;
      const bool in = e >= 0 && e < T.n;
      p[j] = in ? load1<kP>(T.p, e) : 0.0f; g[j] = in ? load1<kG>(T.g, e) : 0.0f;
      m[j] = in ? T.m[e] : 0.0f; v[j] = in ? T.v[e] : 0.0f;
    }
  }
  const float s = a.grad_scale ? *a.grad_scale : 1.0f;
  if (!(fabsf(s) <= 3.402823466e38f)) return;
  const float step_size = a.count ? a.count->step_size : a.step_size;
  const float inv_bc2s = a.count ? a.count->inv_bc2s : a.inv_bc2s;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float gs = __fmul_rn(s, g[j]);
    m[j] = __fadd_rn(__fmul_rn(a.b1, m[j]), __fmul_rn(a.omb1, gs));
    v[j] = __fadd_rn(__fmul_rn(a.b2, v[j]), __fmul_rn(__fmul_rn(a.omb2, gs), gs));
    const float den = __fmaf_rn(__fsqrt_rn(v[j]), inv_bc2s, a.eps);
    p[j] = __fmaf_rn(-step_size, __fdiv_rn(m[j], den), __fmul_rn(p[j], a.decay));
  }
  if (vec) {
    store4<kP>(T.p, i, p); store4<kF32>(T.m, i, m); store4<kF32>(T.v, i, v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t e = i + j * step;
      if (e >= 0 && e < T.n) { store1<kP>(T.p, e, p[j]); T.m[e] = m[j]; T.v[e] = v[j]; }
    }
  }
}

// Two threads, ahead of the step that they count: a bias correction each, in
// binary64 and rounded once, as the host forms them.
__global__ void advance_kernel(StepCount* count, const float* grad_scale, double lr, double b1, double b2) {
  const int64_t taken = count->taken + 1;
  const float s = grad_scale ? *grad_scale : 1.0f;
  if (!(fabsf(s) <= 3.402823466e38f)) return;
  const bool first = threadIdx.x == 0;
  const double bc = 1.0 - pow(first ? b1 : b2, static_cast<double>(taken));
  if (first) {
    count->step_size = static_cast<float>(lr / bc);
  } else {
    count->inv_bc2s = static_cast<float>(1.0 / sqrt(bc));
  }
  __syncwarp(3u);
  if (first) count->taken = taken;
}

// --------------------------------------------------------------------------
// Norm.  A thread sums the squares of four 16-byte pieces in fp32, and such
// sums, and those of the threads, in binary64; each CTA writes its sum to its
// own slot, and the CTA that finishes last adds the slots in order, so the
// result does not depend on the schedule.  Where the pieces' sum leaves the
// range in which fp32 holds it in full (elements above some 1e19 or all below
// 1e-18), they are read again and squared in binary64.  Bound by DRAM: 355M
// bf16 gradients take 116 us (6.1 TB/s), 115.3 without that check.

constexpr int kNormTensors = 1024;
constexpr int kNormCtas = 8;   // per SM
constexpr int kNormPieces = 4;
__host__ __device__ constexpr int norm_chunk(int type) { return kThreads * kNormPieces * (type == BWD_F32 ? 4 : 8); }

struct NormArgs {
  int64_t chunk_start[kNormTensors + 1];
  const void* g[kNormTensors];
  int32_t n_tail[kNormTensors];  // elements of the tensor's last chunk, counted from the 16-byte boundary before it
  uint8_t type[kNormTensors];
  uint8_t shift[kNormTensors];   // elements between that boundary and the tensor's start
  double* slots;                 // one per CTA of all launches of the call
  unsigned int* ticket;          // 0 before the call and after it
  float* factor;
  float* norm;
  int32_t num_tensors;
  int32_t first_slot, total_slots;
  float max_norm, inv_loss_scale;
};

static_assert(sizeof(NormArgs) <= 32764, "kernel parameter space");

__device__ __forceinline__ double block_sum(double x, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
  __syncthreads();
  x = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) x += red[w];
  __syncthreads();
  return x;
}

// The same sum as chunk_squares's in binary64, for the few pieces that need
// it: the square of any fp32 value is an ordinary binary64 number.
template <int kG>
__device__ __noinline__ double chunk_squares_wide(const void* g, int first, int len) {
  constexpr int kVals = kG == kF32 ? 4 : 8;
  double sum = 0.0;
  for (int q = 0; q < kNormPieces; ++q) {
    const int i = (q * kThreads + threadIdx.x) * kVals;
    for (int j = 0; j < kVals; ++j)
      if (i + j >= first && i + j < len) {
        const double x = static_cast<double>(load1<kG>(g, i + j));
        sum = __fma_rn(x, x, sum);
      }
  }
  return sum;
}

// Sum of squares of this thread's share of elements first .. len - 1 of one
// chunk; g is on a 16-byte boundary.
template <int kG>
__device__ __forceinline__ double chunk_squares(const void* g, int first, int len) {
  constexpr int kVals = kG == kF32 ? 4 : 8;  // values of a piece
  uint32_t any = 0;  // bits that are set in any value
  uint4 w[kNormPieces];
#pragma unroll
  for (int q = 0; q < kNormPieces; ++q) {
    const int i = (q * kThreads + threadIdx.x) * kVals;
    w[q] = make_uint4(0u, 0u, 0u, 0u);
    if (i >= first && i + kVals <= len) w[q] = __ldcs(static_cast<const uint4*>(g) + q * kThreads + threadIdx.x);
  }
  float sum[2] = {0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < kNormPieces; ++q) {
    const int i = (q * kThreads + threadIdx.x) * kVals;
    if (i >= first && i + kVals <= len) {
#pragma unroll
      for (int j = 0; j < kVals; ++j) {
        const uint32_t u = (&w[q].x)[kG == kF32 ? j : j / 2];
        any |= u;
        const float x = kG == kF32 ? __uint_as_float(u) : widen<kG>(static_cast<unsigned short>(j % 2 ? u >> 16 : u & 0xffffu));
        sum[j % 2] = __fmaf_rn(x, x, sum[j % 2]);
      }
    } else {
      for (int j = 0; j < kVals; ++j)
        if (i + j >= first && i + j < len) {
          const float x = load1<kG>(g, i + j);
          any |= __float_as_uint(x);
          sum[j % 2] = __fmaf_rn(x, x, sum[j % 2]);
        }
    }
  }
  const float all = __fadd_rn(sum[0], sum[1]);
  // Below 2^-120 the roundings of up to 16 subnormal squares, 2^-150 each, may
  // count.  Squares of fp16 values lie between 2^-48 and 2^32.
  if (kG != kF16 && !(all >= 0x1p-120f && all <= 3.402823466e38f) && (any & (kG == kF32 ? 0x7fffffffu : 0x7fff7fffu)) != 0)
    return chunk_squares_wide<kG>(g, first, len);
  return static_cast<double>(all);
}

__global__ void __launch_bounds__(kThreads, kNormCtas)
grad_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ double s_red[kThreads / 32];
  __shared__ bool s_last;
  const int64_t total = a.chunk_start[a.num_tensors];
  int64_t c = blockIdx.x;
  double part = 0.0;
  if (c < total) {
    int ti = find_tensor(a.chunk_start, a.num_tensors, c);
    for (; c < total; c += gridDim.x) {
      while (a.chunk_start[ti + 1] <= c) ++ti;
      const int type = a.type[ti];
      const int len = c + 1 == a.chunk_start[ti + 1] ? a.n_tail[ti] : norm_chunk(type);
      const int first = c == a.chunk_start[ti] ? a.shift[ti] : 0;
      // a chunk is 64 bytes to a thread, whatever the type
      const char* const g = static_cast<const char*>(a.g[ti]) + (c - a.chunk_start[ti]) * (kThreads * kNormPieces * 16);
      const double sum = type == kF32 ? chunk_squares<kF32>(g, first, len)
                        : type == kBF16 ? chunk_squares<kBF16>(g, first, len) : chunk_squares<kF16>(g, first, len);
      part += sum;
    }
  }
  const double mine = block_sum(part, s_red);
  if (threadIdx.x == 0) {
    a.slots[a.first_slot + blockIdx.x] = mine;
    __threadfence();
    s_last = atomicAdd(a.ticket, 1u) + 1u == static_cast<unsigned int>(a.total_slots);
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  double all = 0.0;
  for (int i = threadIdx.x; i < a.total_slots; i += kThreads) all += __ldcg(a.slots + i);
  all = block_sum(all, s_red);
  if (threadIdx.x == 0) {
    const float norm = static_cast<float>(sqrt(all) * static_cast<double>(a.inv_loss_scale));
    const float clip = fminf(1.0f, __fdiv_rn(a.max_norm, __fadd_rn(norm, 1e-6f)));
    const bool finite = norm <= 3.402823466e38f;  // false for NaN too
    *a.factor = finite ? __fmul_rn(clip, a.inv_loss_scale) : __uint_as_float(0x7fffffffu);
    *a.norm = norm;
    *a.ticket = 0;
  }
}

// --------------------------------------------------------------------------
// host side

bwd_status sm_count(int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? BWD_OK : cuda_fail(e, "cudaDeviceGetAttribute");
}

int64_t chunks_of(int64_t n, int64_t chunk) { return (n + chunk - 1) / chunk; }
bool valid_type(int t) { return t == BWD_F32 || t == BWD_BF16 || t == BWD_F16; }
uintptr_t bytes_of(int t) { return t == BWD_F32 ? 4 : 2; }

// Elements between a pointer and the boundary of four of them before it.
int64_t past_quad(const void* x, int type) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(x) / bytes_of(type) % 4); }

bwd_status launch_adam32(const Adam32Args& a, int g_type, int p_type, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.chunk_start[a.num_tensors]);
  switch (3 * p_type + g_type) {
    case 0: adam32_kernel<kF32, kF32><<<grid, kThreads, 0, st>>>(a); break;
    case 1: adam32_kernel<kBF16, kF32><<<grid, kThreads, 0, st>>>(a); break;
    case 2: adam32_kernel<kF16, kF32><<<grid, kThreads, 0, st>>>(a); break;
    case 3: adam32_kernel<kF32, kBF16><<<grid, kThreads, 0, st>>>(a); break;
    case 4: adam32_kernel<kBF16, kBF16><<<grid, kThreads, 0, st>>>(a); break;
    case 5: adam32_kernel<kF16, kBF16><<<grid, kThreads, 0, st>>>(a); break;
    case 6: adam32_kernel<kF32, kF16><<<grid, kThreads, 0, st>>>(a); break;
    case 7: adam32_kernel<kBF16, kF16><<<grid, kThreads, 0, st>>>(a); break;
    default: adam32_kernel<kF16, kF16><<<grid, kThreads, 0, st>>>(a); break;
  }
  return check_launch("adam32_kernel launch");
}

// The step of either entry point; with `count`, hp's step is not read.
bwd_status adam32_step(int32_t num_tensors, void* const* p, bwd_dtype p_dtype, const void* const* g, bwd_dtype g_dtype,
                       float* const* m, float* const* v, const int64_t* n, const float* grad_scale, StepCount* count,
                       const bwd_adamw_hparams* hp, void* stream) {
  if (num_tensors < 0) return fail(BWD_ERR_INVALID_ARG, "num_tensors < 0");
  if (!valid_type(g_dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "gradient dtype %d", (int)g_dtype);
  if (!valid_type(p_dtype)) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "parameter dtype %d", (int)p_dtype);
  bwd_status s = bwd::host::check_hparams(hp);
  if (s != BWD_OK) return s;
  if (num_tensors == 0) return BWD_OK;
  if (!p || !g || !m || !v || !n) return fail(BWD_ERR_INVALID_ARG, "NULL array");
  if (!aligned_to(grad_scale, 4)) return fail(BWD_ERR_INVALID_ARG, "grad_scale is not 4-byte aligned");
  for (int32_t i = 0; i < num_tensors; ++i) {
    if (n[i] < 0 || n[i] > (kMaxChunks - 1) * kChunk) return fail(BWD_ERR_INVALID_ARG, "tensor %d: bad size", i);
    if (n[i] > 0 && (!p[i] || !g[i] || !m[i] || !v[i])) return fail(BWD_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
    if (n[i] > 0 && (!aligned_to(p[i], bytes_of(p_dtype)) || !aligned_to(g[i], bytes_of(g_dtype)) ||
                     !aligned_to(m[i], 4) || !aligned_to(v[i], 4)))
      return fail(BWD_ERR_INVALID_ARG, "tensor %d: pointer not aligned to its element size", i);
  }
  if (count && (s = bwd::host::advance(count, grad_scale, *hp, stream)) != BWD_OK) return s;
  static thread_local Adam32Args a;  // ~27 KB: kept off the stack
  const bwd::host::AdamScalars k = bwd::host::adam_scalars(*hp);
  a.b1 = k.b1; a.omb1 = k.omb1; a.b2 = k.b2; a.omb2 = k.omb2;
  a.eps = k.eps; a.step_size = k.step_size; a.inv_bc2s = k.inv_bc2s; a.decay = k.decay;
  a.grad_scale = grad_scale;
  a.count = count;
  a.chunk_start[0] = 0;
  int t = 0;
  const auto flush = [&] {
    if (t == 0) return BWD_OK;
    a.num_tensors = t;
    t = 0;
    return launch_adam32(a, g_dtype, p_dtype, static_cast<cudaStream_t>(stream));
  };
  for (int32_t i = 0; i < num_tensors; ++i) {
    if (n[i] == 0) continue;
    const int64_t at[4] = {past_quad(p[i], p_dtype), past_quad(g[i], g_dtype), past_quad(m[i], BWD_F32), past_quad(v[i], BWD_F32)};
    const int64_t shift = at[0] == at[1] && at[0] == at[2] && at[0] == at[3] ? at[0] : -1;
    const int64_t chunks = chunks_of(n[i] + (shift > 0 ? shift : 0), kChunk);
    if (t == kMaxTensors || a.chunk_start[t] + chunks > kMaxChunks)
      if ((s = flush()) != BWD_OK) return s;
    a.t[t] = Tensor32{p[i], g[i], m[i], v[i], n[i], shift};
    a.chunk_start[t + 1] = a.chunk_start[t] + chunks;
    ++t;
  }
  return flush();
}

}  // namespace

namespace bwd {
namespace host {

bwd_status advance(StepCount* count, const float* grad_scale, const bwd_adamw_hparams& hp, void* stream) {
  advance_kernel<<<1, 2, 0, static_cast<cudaStream_t>(stream)>>>(count, grad_scale, hp.lr, hp.beta1, hp.beta2);
  return check_launch("advance_kernel launch");
}

}  // namespace host
}  // namespace bwd

extern "C" {

bwd_status bwd_adam32_step_multi(int32_t num_tensors, void* const* p, bwd_dtype p_dtype, const void* const* g,
                                 bwd_dtype g_dtype, float* const* m, float* const* v, const int64_t* n,
                                 const float* grad_scale, const bwd_adamw_hparams* hp, void* stream) {
  return adam32_step(num_tensors, p, p_dtype, g, g_dtype, m, v, n, grad_scale, nullptr, hp, stream);
}

bwd_status bwd_adam32_step_multi_counted(int32_t num_tensors, void* const* p, bwd_dtype p_dtype, const void* const* g,
                                         bwd_dtype g_dtype, float* const* m, float* const* v, const int64_t* n,
                                         const float* grad_scale, void* count, const bwd_adamw_hparams* hp, void* stream) {
  if (!count || !aligned_to(count, 8)) return fail(BWD_ERR_INVALID_ARG, "count is NULL or not 8-byte aligned");
  if (!hp) return fail(BWD_ERR_INVALID_ARG, "hparams is NULL");
  bwd_adamw_hparams h = *hp;
  h.step = 1;
  return adam32_step(num_tensors, p, p_dtype, g, g_dtype, m, v, n, grad_scale, static_cast<StepCount*>(count), &h, stream);
}

int64_t bwd_grad_norm_work_bytes(int32_t num_tensors) {
  if (num_tensors < 0) return -1;
  // a ticket, and a slot for each CTA of each launch, of which a call over no
  // tensor has one too; 256 SMs are more than the device has
  const int64_t launches = num_tensors > kNormTensors ? (static_cast<int64_t>(num_tensors) + kNormTensors - 1) / kNormTensors : 1;
  return 16 + 8 * launches * 256 * kNormCtas;
}

bwd_status bwd_grad_norm(int32_t num_tensors, const void* const* g, const int32_t* g_dtype, const int64_t* n, float max_norm,
                         float loss_scale, float* factor, float* norm, void* work, void* stream) {
  if (num_tensors < 0) return fail(BWD_ERR_INVALID_ARG, "num_tensors < 0");
  if (!(max_norm > 0.0f)) return fail(BWD_ERR_INVALID_ARG, "max_norm must be > 0");
  if (!(loss_scale > 0.0f) || !std::isfinite(loss_scale) || !std::isfinite(1.0f / loss_scale))
    return fail(BWD_ERR_INVALID_ARG, "loss_scale and its reciprocal must be finite and > 0");
  if (!factor || !norm || !work || (num_tensors > 0 && (!g || !g_dtype || !n))) return fail(BWD_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned_to(factor, 4) || !aligned_to(norm, 4) || !aligned16(work))
    return fail(BWD_ERR_INVALID_ARG, "factor and norm must be 4-byte and work 16-byte aligned");
  for (int32_t i = 0; i < num_tensors; ++i) {
    if (n[i] < 0) return fail(BWD_ERR_INVALID_ARG, "tensor %d: n < 0", i);
    if (!valid_type(g_dtype[i])) return fail(BWD_ERR_UNSUPPORTED_DTYPE, "tensor %d: gradient dtype %d", i, (int)g_dtype[i]);
    if (n[i] > 0 && (!g[i] || !aligned_to(g[i], bytes_of(g_dtype[i]))))
      return fail(BWD_ERR_INVALID_ARG, "tensor %d: NULL or unaligned pointer", i);
  }
  int sms = 0;
  bwd_status s = sm_count(&sms);
  if (s != BWD_OK) return s;
  static thread_local NormArgs a;  // ~20 KB: kept off the stack
  a.ticket = static_cast<unsigned int*>(work);
  a.slots = reinterpret_cast<double*>(static_cast<char*>(work) + 16);
  a.factor = factor;
  a.norm = norm;
  a.max_norm = max_norm;
  a.inv_loss_scale = 1.0f / loss_scale;
  const int64_t cap = static_cast<int64_t>(sms < 256 ? sms : 256) * kNormCtas;
  // two passes: how many CTAs all launches have together, then the launches;
  // one pass where there is one launch
  int64_t slots = 0;
  for (int pass = num_tensors > kNormTensors ? 0 : 1; pass < 2; ++pass) {
    int64_t first = 0;
    int t = 0;
    a.chunk_start[0] = 0;
    for (int32_t i = 0; i <= num_tensors; ++i) {
      if (i < num_tensors && n[i] > 0) {
        const uintptr_t over = reinterpret_cast<uintptr_t>(g[i]) % 16;
        const int64_t shift = static_cast<int64_t>(over / bytes_of(g_dtype[i]));
        const int64_t chunk = norm_chunk(g_dtype[i]), chunks = chunks_of(n[i] + shift, chunk);
        a.g[t] = static_cast<const char*>(g[i]) - over;
        a.type[t] = static_cast<uint8_t>(g_dtype[i]);
        a.shift[t] = static_cast<uint8_t>(shift);
        a.n_tail[t] = static_cast<int32_t>(n[i] + shift - (chunks - 1) * chunk);
        a.chunk_start[t + 1] = a.chunk_start[t] + chunks;
        ++t;
      }
      // the last launch may have no tensors: it still forms the result
      if (t == kNormTensors || (i == num_tensors && (t > 0 || first == 0))) {
        const int64_t chunks = a.chunk_start[t], ctas = chunks < 1 ? 1 : chunks < cap ? chunks : cap;
        if (pass == 1) {
          a.num_tensors = t;
          a.first_slot = static_cast<int32_t>(first);
          a.total_slots = static_cast<int32_t>(slots ? slots : ctas);
          cudaStream_t st = static_cast<cudaStream_t>(stream);
          const int grid = static_cast<int>(ctas);
          grad_norm_kernel<<<grid, kThreads, 0, st>>>(a);
          if ((s = check_launch("grad_norm_kernel launch")) != BWD_OK) return s;
        }
        first += ctas;
        t = 0;
      }
    }
    slots = first;
  }
  return BWD_OK;
}

}  // extern "C"
