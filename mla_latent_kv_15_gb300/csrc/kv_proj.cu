// Latent rows to every head's key and value (mla_kv_up_proj), on tcgen05:
//
//   kv[t, c] = sum_l latent[t, l] * w[c, l]      l < 512, c = n * D + d
//
// one product of [T, 512] with [C, 512]^T, both operands K-major.  float32
// accumulation in tensor memory, one rounding to bf16.
//
// Few tokens (kv_proj_kernel): the weights are the traffic.  One CTA computes
// a 128-token x bn-column tile; its ring holds as much of the 512-deep
// contraction as the shared memory of half an SM does, so nearly every load
// of a CTA is in flight at once.  With fewer than 128 tokens the token box
// holds only round_up(T, 16) rows; the MMA rows past it read other bytes of
// the CTA's shared memory and their results are never stored.
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {
using namespace ptx;

constexpr int kM = 128;                          // tokens per CTA (MMA M)
constexpr int kK = 64;                           // contraction dims per stage: one 128-byte swizzled row
constexpr int kChunks = kLkv / kK;               // 8
constexpr int kThreads = 192;                    // TMA warp, MMA warp, 4 epilogue warps
constexpr uint32_t kXBoxMax = kM * kK * 2;       // 16 KB
constexpr uint32_t kRingBudget = 96 * 1024;      // two CTAs share an SM
constexpr uint32_t kSmemPerSm = 233472;

__device__ unsigned int g_kv_proj_error;         // OR of MLA_DEVERR_* bits (read by mla_proj_status)

struct Bars {
  uint64_t full[kChunks];
  uint64_t empty[kChunks];
  uint64_t d_full;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void give_up(Bars* bars) {
  atomicOr(&g_kv_proj_error, 1u);  // MLA_DEVERR_TIMEOUT
  *reinterpret_cast<volatile int*>(&bars->abort) = 1;
}

// 32 accumulator columns of a row as bf16, at column c0 of the row `dst`; columns at or past C are left out.
__device__ __forceinline__ void store_cols32(__nv_bfloat16* dst, const uint32_t (&r)[32], int64_t c0, int64_t C) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (c0 + 8 * v < C)
      *reinterpret_cast<uint4*>(dst + 8 * v) =
          make_uint4(pack_bf16x2(__uint_as_float(r[8 * v]), __uint_as_float(r[8 * v + 1])),
                     pack_bf16x2(__uint_as_float(r[8 * v + 2]), __uint_as_float(r[8 * v + 3])),
                     pack_bf16x2(__uint_as_float(r[8 * v + 4]), __uint_as_float(r[8 * v + 5])),
                     pack_bf16x2(__uint_as_float(r[8 * v + 6]), __uint_as_float(r[8 * v + 7])));
}

__global__ void __launch_bounds__(kThreads, 1)
    kv_proj_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   __nv_bfloat16* __restrict__ y, int64_t T, int64_t C, int bn, int stages, int xrows) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t xbox = (uint32_t)xrows * kK * 2, wbox = (uint32_t)bn * kK * 2;
  const uint32_t stage_bytes = xbox + wbox;
  Bars* bars = reinterpret_cast<Bars*>(smem + stages * stage_bytes + (kXBoxMax - xbox));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x * bn, t0 = blockIdx.y * kM;
  const uint32_t tcols = bn <= 64 ? 64 : bn <= 128 ? 128 : 256;
  const int npre = stages < kChunks ? stages : kChunks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->d_full), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    // a programmatic dependent: what is above overlaps the previous kernel,
    // whose output the operands may be
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int c = 0; c < npre; ++c) {
      const uint32_t st = smem_u32(smem + c * stage_bytes), full = smem_u32(&bars->full[c]);
      mbar_expect_tx(full, stage_bytes);
      tma_load_2d(st, &tm_x, c * kK, t0, full);
      tma_load_2d(st + xbox, &tm_w, c * kK, c0, full);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    if (lane == 0) {
      int issued = npre;
      for (int c = npre; c < kChunks; ++c) {
        const int slot = c % stages, round = c / stages;
        if (!mbar_wait(smem_u32(&bars->empty[slot]), (round - 1) & 1)) {
          give_up(bars);
          break;
        }
        if (*abort_flag) break;
        const uint32_t st = smem_u32(smem + slot * stage_bytes), full = smem_u32(&bars->full[slot]);
        mbar_expect_tx(full, stage_bytes);
        tma_load_2d(st, &tm_x, c * kK, t0, full);
        tma_load_2d(st + xbox, &tm_w, c * kK, c0, full);
        issued = c + 1;
      }
      // every copy this thread issued has landed before the CTA may exit
      for (int c = issued > stages ? issued - stages : 0; c < issued; ++c)
        if (!mbar_wait(smem_u32(&bars->full[c % stages]), (c / stages) & 1)) give_up(bars);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kM, bn, 0, 0);
      for (int c = 0; c < kChunks; ++c) {
        const int slot = c % stages;
        if (!mbar_wait(smem_u32(&bars->full[slot]), (c / stages) & 1)) {
          give_up(bars);
          break;
        }
        if (*abort_flag) break;
        tc_fence_after();
        const uint32_t st = smem_u32(smem + slot * stage_bytes);
        const uint64_t xd = smem_desc(st, 16, 1024, kSwizzle128B);
        const uint64_t wd = smem_desc(st + xbox, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < kK / 16; ++k)
          mma_ss(tmem, xd + ((k * 32) >> 4), wd + ((k * 32) >> 4), idesc, (c > 0 || k > 0) ? 1u : 0u);
        mma_commit(smem_u32(&bars->empty[slot]));
      }
      mma_commit(smem_u32(&bars->d_full));
      if (!mbar_wait(smem_u32(&bars->d_full), 0)) give_up(bars);
    }
  } else {
    const int q = warp & 3;
    const int64_t t = t0 + 32 * q + lane;
    const bool done = mbar_wait(smem_u32(&bars->d_full), 0);
    if (!done) give_up(bars);
    tc_fence_after();
    if (done && !*abort_flag) {
      __nv_bfloat16* dst = y + t * C + c0;
      for (int j = 0; j < bn; j += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + j, r);
        tmem_wait_ld();
        if (t < T) store_cols32(dst + j, r, c0 + j, C);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

}  // namespace

KvProjShape kv_proj_shape(int64_t T, int64_t C, int sms) {
  KvProjShape p{};
  p.bn = 128;
  p.xrows = T >= kM ? kM : (int)((T + 15) / 16 * 16);
  (void)C, (void)sms;
  return p;
}

cudaError_t launch_kv_proj(const CUtensorMap& tm_x, const CUtensorMap& tm_w, void* y, int64_t T, int64_t C,
                           const KvProjShape& p, cudaStream_t s) {
  const uint32_t xbox = (uint32_t)p.xrows * kK * 2, stage = xbox + (uint32_t)p.bn * kK * 2;
  int stages = (int)(kRingBudget / stage);
  if (stages > kChunks) stages = kChunks;
  size_t smem = 1024 + (size_t)stages * stage + (kXBoxMax - xbox) + sizeof(Bars);
  // never more CTAs on an SM than its 512 tensor-memory columns hold (an
  // allocation beyond them would wait for another CTA to finish)
  const uint32_t tcols = p.bn <= 64 ? 64 : p.bn <= 128 ? 128 : 256;
  const size_t floor_smem = kSmemPerSm / (512 / tcols + 1);
  if (smem < floor_smem) smem = floor_smem;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kv_proj_kernel, 1024 + kRingBudget + kXBoxMax + sizeof(Bars) + 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((C + p.bn - 1) / p.bn), (unsigned)((T + kM - 1) / kM));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_proj_kernel, tm_x, tm_w, static_cast<__nv_bfloat16*>(y), T, C, p.bn, stages,
                         p.xrows);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t kv_proj_status(int* status, int clear, cudaStream_t s) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_kv_proj_error, sizeof v, 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_kv_proj_error, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  *status = (int)v;
  return e;
}

}  // namespace mla
