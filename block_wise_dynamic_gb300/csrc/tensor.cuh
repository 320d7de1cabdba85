// What the translation units of matrix products and their neighbours share:
// conversions, barriers with bounded waits, tensor copies and tensor memory,
// and on the host tensor maps, launches and workspaces.
#pragma once

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
using bwd::host::cuda_fail;
using bwd::host::fail;

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

template <int kT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if (kT == kF32) return static_cast<const float*>(x)[i];
  const unsigned short h = static_cast<const unsigned short*>(x)[i];
  if (kT == kBF16) return __uint_as_float(static_cast<uint32_t>(h) << 16);
  return __half2float(__ushort_as_half(h));
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

// --------------------------------------------------------------------------
// barriers, copies and tensor memory

__device__ unsigned int g_wait_fault;  // set when a bounded wait gives up

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
  atomicOr(&g_wait_fault, 1u);
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

// The largest of 8, 4 and 2 bytes that divides a matrix's address and row.
int unit_of(const void* base, int64_t row_bytes) {
  return aligned_to(base, 8) && row_bytes % 8 == 0 ? 8 : aligned_to(base, 4) && row_bytes % 4 == 0 ? 4 : 2;
}

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

template <typename F>
cudaError_t opt_in(F* kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
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

// Reads and clears this translation unit's fault word.
[[maybe_unused]] bwd_status take_wait_fault(unsigned int* fault) {
  cudaError_t e = cudaMemcpyFromSymbol(fault, g_wait_fault, sizeof *fault);
  if (e != cudaSuccess) return cuda_fail(e, "cudaMemcpyFromSymbol(fault word)");
  if (*fault == 0) return BWD_OK;
  const unsigned int zero = 0;
  e = cudaMemcpyToSymbol(g_wait_fault, &zero, sizeof zero);
  return e == cudaSuccess ? BWD_OK : cuda_fail(e, "cudaMemcpyToSymbol(fault word)");
}

}  // namespace
