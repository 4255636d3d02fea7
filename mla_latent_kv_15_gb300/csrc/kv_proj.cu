// Latent rows to every head's key and value (mla_kv_up_proj), on tcgen05:
//
//   kv[t, c] = sum_l latent[t, l] * w[c, l]      l < 512, c = n * D + d
//
// one product of [T, 512] with [C, 512]^T, both operands K-major.  float32
// accumulation in tensor memory, one rounding to bf16.
//
// Few tokens (kv_proj_kernel): the weights are the traffic.  One CTA computes
// a 128-token x kBN-column tile; its ring holds as much of the 512-deep
// contraction as the shared memory of half an SM does, so nearly every load
// of a CTA is in flight at once.  With fewer than 128 tokens the token box
// holds only round_up(T, 16) rows; the MMA rows past it read other bytes of
// the CTA's shared memory and their results are never stored.
//
// Many tokens (kv_proj_pair_kernel): CTA pairs walk 256-token x kBN-column
// tiles (cta_group::2: each CTA holds 128 tokens and half the columns of a
// stage), two accumulators in tensor memory, so that the stores of a tile run
// under the products of the next.  The epilogue leaves in 32-row x 64-column
// pieces staged in shared memory and stored by TMA, which clips ragged edges.
// What bounds it is the loads' latency beside the stores (8192 tokens x 32768
// columns: 136 us without the stores): shared memory goes to load stages, and
// two staged pieces a warp are enough (pieces 2, 4, 6, 8, leaving 6, 5, 4, 3
// stages: 174, 181, 186, 200 us; the tokens kept in shared memory and only
// weights streamed, four stages: 212; 32-byte stores from registers: 202).
// Without the graph's launch 173 us back to back in a long run: 1590 TFLOP/s, 83 % of the
// library's burst rate and 94 % of its sustained one.
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

template <int kBN>
__global__ void __launch_bounds__(kThreads, 1)
    kv_proj_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   __nv_bfloat16* __restrict__ y, int64_t T, int64_t C, int stages, int xrows) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr uint32_t wbox = kBN * kK * 2;
  const uint32_t xbox = (uint32_t)xrows * kK * 2;
  const uint32_t stage_bytes = xbox + wbox;
  Bars* bars = reinterpret_cast<Bars*>(smem + stages * stage_bytes + (kXBoxMax - xbox));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.x * kBN, t0 = blockIdx.y * kM;
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
    tmem_alloc(smem_u32(&bars->tmem_base), kBN);
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
    const uint32_t idesc = idesc_bf16_f32(kM, kBN, 0, 0);
    for (int c = 0; c < kChunks; ++c) {
      const int slot = c % stages;
      if (!mbar_wait(smem_u32(&bars->full[slot]), (c / stages) & 1)) {
        give_up(bars);
        break;
      }
      if (*abort_flag) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t st = smem_u32(smem + slot * stage_bytes);
        const uint64_t xd = smem_desc(st, 16, 1024, kSwizzle128B);
        const uint64_t wd = smem_desc(st + xbox, 16, 1024, kSwizzle128B);
#pragma unroll
        for (int k = 0; k < kK / 16; ++k)
          mma_ss(tmem, xd + ((k * 32) >> 4), wd + ((k * 32) >> 4), idesc, (c > 0 || k > 0) ? 1u : 0u);
        mma_commit(smem_u32(&bars->empty[slot]));
        if (c == kChunks - 1) mma_commit(smem_u32(&bars->d_full));
      }
      __syncwarp();
    }
    if (!*abort_flag && !mbar_wait(smem_u32(&bars->d_full), 0)) give_up(bars);
    __syncwarp();
  } else {
    const int q = warp & 3;
    const int64_t t = t0 + 32 * q + lane;
    const bool done = mbar_wait(smem_u32(&bars->d_full), 0);
    if (!done) give_up(bars);
    tc_fence_after();
    if (done && !*abort_flag) {
      __nv_bfloat16* dst = y + t * C + c0;
      for (int j = 0; j < kBN; j += 32) {
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
    tmem_dealloc(tmem, kBN);
  }
}

// ------------------------------------------------------------- many tokens

constexpr int kPairThreads = 192;                // load warp, MMA warp, 4 epilogue warps
constexpr uint32_t kPiece = 32 * 128;            // 32 rows x 64 bf16

constexpr int kPieces = 2;                       // staged pieces of an epilogue warp

template <int kBN>
struct PairShape {
  static constexpr uint32_t kTmem = kBN <= 128 ? 256 : 512;   // columns: two accumulators, a power of two
  static constexpr uint32_t kWBox = kBN / 2 * kK * 2;
  static constexpr uint32_t kStage = kXBoxMax + kWBox;
  static constexpr uint32_t kStaging = 4 * kPieces * kPiece;
  static constexpr int kStages = (int)((232448 - 1024 - 512 - kStaging) / kStage) < 8
                                     ? (int)((232448 - 1024 - 512 - kStaging) / kStage)
                                     : 8;
  static constexpr size_t kSmem = 1024 + kStages * kStage + kStaging + 512;
};

// Barriers marked (lead) are used in the leading CTA only, by both CTAs.
struct PairBars {
  uint64_t full[8];        // (lead) both CTAs' boxes have landed
  uint64_t empty[8];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];   // (lead) the epilogue warps of both CTAs
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(PairBars) <= 512, "fits behind the staging");

__device__ __forceinline__ void pair_wait(PairBars* bars, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait(at, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_hint(at, parity, kWaitHintNs)) {
    if (*(volatile int*)&bars->abort) return;
    if (globaltimer() - t0 > MLA_WAIT_LIMIT_NS) {
      *(volatile int*)&bars->abort = 1;
      atomicOr(&g_kv_proj_error, 1u);  // MLA_DEVERR_TIMEOUT
      return;
    }
  }
}

template <int kBN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    kv_proj_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                        const __grid_constant__ CUtensorMap tm_y, int T, int C, int tiles_m, int tiles_n) {
  using P = PairShape<kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* staging = smem + P::kStages * P::kStage;
  PairBars* bars = reinterpret_cast<PairBars*>(staging + P::kStaging);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int first = (int)cluster_id_x(), step = gridDim.x / 2, tiles = tiles_m * tiles_n;
  volatile int* abort_flag = &bars->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 2);
      mbar_init(smem_u32(&bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->acc_full[i]), 1);
      mbar_init(smem_u32(&bars->acc_empty[i]), 8);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_y);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&bars->tmem_base), P::kTmem);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are initialised before either uses the other's
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // tile i: the token tiles of a column tile follow one another (its weights stay in L2, all tokens do)
  if (warp == 0) {
    uint32_t n = 0;
    for (int i = first; i < tiles && !*abort_flag; i += step) {
      const int t0 = (i % tiles_m) * 256 + 128 * (int)rank, c0 = (i / tiles_m) * kBN + kBN / 2 * (int)rank;
      for (int c = 0; c < kChunks; ++c, ++n) {
        const uint32_t slot = n % P::kStages;
        pair_wait(bars, &bars->empty[slot], ((n / P::kStages) & 1) ^ 1);
        if (*abort_flag) break;
        if (elect_one()) {
          const uint32_t st = smem_u32(smem + slot * P::kStage), full = mapa(smem_u32(&bars->full[slot]), 0);
          mbar_expect_tx_remote(full, P::kStage);
          tma_load_2d_pair(st, &tm_x, c * kK, t0, full);
          tma_load_2d_pair(st + kXBoxMax, &tm_w, c * kK, c0, full);
        }
        __syncwarp();
      }
    }
    // every load of the pair has landed before it ends
    if (rank == 0)
      for (uint32_t k = n > P::kStages ? n - P::kStages : 0; k < n; ++k)
        pair_wait(bars, &bars->full[k % P::kStages], (k / P::kStages) & 1);
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(256, kBN, 0, 0);
      constexpr uint32_t hi = desc_hi(1024, kSwizzle128B);
      const uint32_t x_lo = desc_lo(smem_u32(smem), 16), w_lo = desc_lo(smem_u32(smem) + kXBoxMax, 16);
      uint32_t n = 0, m = 0;
      for (int i = first; i < tiles && !*abort_flag; i += step, ++m) {
        const uint32_t acc = m & 1;
        pair_wait(bars, &bars->acc_empty[acc], ((m >> 1) & 1) ^ 1);
        tc_fence_after();
        for (int c = 0; c < kChunks; ++c, ++n) {
          const uint32_t slot = n % P::kStages;
          pair_wait(bars, &bars->full[slot], (n / P::kStages) & 1);
          if (elect_one()) {
            const uint32_t off = slot * (P::kStage >> 4);
#pragma unroll
            for (int k = 0; k < kK / 16; ++k)
              mma_pair_ss(tmem + acc * kBN, x_lo + off + 2 * k, hi, w_lo + off + 2 * k, hi, idesc, (c | k) ? 1u : 0u);
            mma_commit_pair(smem_u32(&bars->empty[slot]));
            if (c == kChunks - 1) mma_commit_pair(smem_u32(&bars->acc_full[acc]));
          }
          __syncwarp();
        }
      }
      if (elect_one()) mma_commit_pair(smem_u32(&bars->drain));
      __syncwarp();
      pair_wait(bars, &bars->drain, 0);   // every product of the pair is done
    }
  } else {
    const int q = warp & 3;
    uint8_t* stage = staging + q * kPieces * kPiece;
    uint32_t m = 0;
    for (int i = first; i < tiles && !*abort_flag; i += step, ++m) {
      const uint32_t acc = m & 1;
      const int t0 = (i % tiles_m) * 256 + 128 * (int)rank + 32 * q, c0 = (i / tiles_m) * kBN;
      pair_wait(bars, &bars->acc_full[acc], (m >> 1) & 1);
      if (*abort_flag) break;
      tc_fence_after();
      const uint32_t from = tmem + acc * kBN + ((uint32_t)(32 * q) << 16);
#pragma unroll 1
      for (int p = 0; p < kBN / 64; ++p) {
        uint8_t* piece = stage + (m * (kBN / 64) + p) % kPieces * kPiece;   // the pieces in turn, across tiles
        uint32_t a[32], b[32];
        tmem_ld32(from + 64 * p, a);
        tmem_ld32(from + 64 * p + 32, b);
        // the piece's last store has read it
        if (lane == 0) bulk_wait_group_read<kPieces - 1>();
        tmem_wait_ld();
        __syncwarp();
        const uint32_t row = smem_u32(piece) + lane * 128;
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = 8 * (v & 3) + 2 * e;
            w[e] = v < 4 ? pack_bf16x2(__uint_as_float(a[k]), __uint_as_float(a[k + 1]))
                         : pack_bf16x2(__uint_as_float(b[k]), __uint_as_float(b[k + 1]));
          }
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((v ^ (lane & 7)) << 4)), "r"(w[0]),
                       "r"(w[1]), "r"(w[2]), "r"(w[3])
                       : "memory");
        }
        if (p == kBN / 64 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&bars->acc_empty[acc]), 0));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (t0 < T && c0 + 64 * p < C) tma_store_2d(&tm_y, c0 + 64 * p, t0, smem_u32(piece));
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  if (*abort_flag) {
    // given up: loads and products in flight finish well within this time
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // the pair ends together: each reads and signals the other's shared memory
  if (warp == 1) {
    // the last signal to the peer's own barriers is on its way by now (awaited
    // from the kernel's start, the wait would bound the whole call)
    if (rank == 1) pair_wait(bars, &bars->drain, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, P::kTmem);
  }
}

template <int kBN>
cudaError_t launch_pair(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_y, int64_t T,
                        int64_t C, int pairs, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kv_proj_pair_kernel<kBN>, PairShape<kBN>::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t tm = (T + 255) / 256, tn = (C + kBN - 1) / kBN;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (tm * tn < pairs ? tm * tn : pairs)));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = PairShape<kBN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_proj_pair_kernel<kBN>, tm_x, tm_w, tm_y, (int)T, (int)C, (int)tm, (int)tn);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int kBN>
cudaError_t launch_few(const CUtensorMap& tm_x, const CUtensorMap& tm_w, void* y, int64_t T, int64_t C, int xrows,
                       cudaStream_t s) {
  const uint32_t xbox = (uint32_t)xrows * kK * 2, stage = xbox + kBN * kK * 2;
  int stages = (int)(kRingBudget / stage);
  if (stages > kChunks) stages = kChunks;
  size_t smem = 1024 + (size_t)stages * stage + (kXBoxMax - xbox) + sizeof(Bars);
  // never more CTAs on an SM than its 512 tensor-memory columns hold (an
  // allocation beyond them would wait for another CTA to finish)
  constexpr size_t floor_smem = kSmemPerSm / (512 / kBN + 1);
  if (smem < floor_smem) smem = floor_smem;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(kv_proj_kernel<kBN>, 1024 + kRingBudget + kXBoxMax + sizeof(Bars) + 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((C + kBN - 1) / kBN), (unsigned)((T + kM - 1) / kM));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_proj_kernel<kBN>, tm_x, tm_w, static_cast<__nv_bfloat16*>(y), T, C, stages,
                         xrows);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

// Up to 128 tokens a single CTA's tile holds them all and the weights' traffic
// wants many CTAs: 32 columns each while that makes no more CTAs than SMs, for
// the shorter products and stores, else 128.  Measured, us a launch among others
// in a graph, weights in L2:  32 columns   128
//    37 tokens x 4096                4.2   4.6
//   128        x 4096                4.2   5.2
//    37        x 5120 (160 CTAs)     4.9   4.7
//    64        x 32768              17.7   8.7
// Above, pairs: 128, 192 or 256 columns a tile, whichever costs least: the
// rounds of all pairs at 100 : 120 : 140 (the wider tile reads less for a
// product), and 45 and 70 for the last stores of the wider ones.  Constants from
// 85 drawn shapes (129 to 8192 tokens, 256 to 32768 columns, weights from L2 and
// from HBM), where the choice takes 0.1 % longer than the best width on average
// and 3.8 % at most; on 60 others 0.04 % and 1.8 %.  One width for all would take
// 7 % (128), 8 % (192) or 11 % (256) longer on average.  Some shapes, us a launch
// as above in short bursts, rounds in brackets:
//                   128         192         256
//   200 x 16384    6.6 (2)     7.9 (2)     7.3 (1)
//  1021 x  5120    8.1 (3)     7.2 (2)     8.4 (2)
//  2048 x 10240   21.4 (9)    18.7 (6)    19.5 (5)
//  4096 x  4096   17.5 (7)    16.4 (5)    15.9 (4)
//  5386 x  7168   33.1 (17)   30.9 (11)   28.8 (9)
//  8192 x 32768    206 (108)   183 (72)    168 (54)    (long runs, under the power cap: 173 to 187)
KvProjShape kv_proj_shape(int64_t T, int64_t C, int sms) {
  KvProjShape p{};
  p.pairs = sms / 2;
  if (T > kM && p.pairs > 0) {
    auto rounds = [&](int bn) { return ((T + 255) / 256 * ((C + bn - 1) / bn) + p.pairs - 1) / p.pairs; };
    const int64_t c128 = 100 * rounds(128), c192 = 120 * rounds(192) + 45, c256 = 140 * rounds(256) + 70;
    p.pair_bn = c128 <= c192 && c128 <= c256 ? 128 : c192 < c256 ? 192 : 256;
    p.wrows = p.pair_bn / 2;
    p.xrows = kM;
  } else {
    p.bn = p.wrows = (C + 31) / 32 <= sms ? 32 : 128;
    p.xrows = T >= kM ? kM : (int)((T + 15) / 16 * 16);
  }
  return p;
}

cudaError_t launch_kv_proj(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_y, void* y,
                           int64_t T, int64_t C, const KvProjShape& p, cudaStream_t s) {
  if (p.pair_bn == 256) return launch_pair<256>(tm_x, tm_w, tm_y, T, C, p.pairs, s);
  if (p.pair_bn == 192) return launch_pair<192>(tm_x, tm_w, tm_y, T, C, p.pairs, s);
  if (p.pair_bn == 128) return launch_pair<128>(tm_x, tm_w, tm_y, T, C, p.pairs, s);
  if (p.bn == 32) return launch_few<32>(tm_x, tm_w, y, T, C, p.xrows, s);
  return launch_few<128>(tm_x, tm_w, y, T, C, p.xrows, s);
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
