// In-place compaction of requests' cache rows (mla_cache_compact): row keep[i]
// of a request to its row i, and its accumulated weight with it.
//
// keep[i] >= i, so a row is only ever moved towards the front.  A request
// belongs to one cluster of CTAs, which walks its rows in waves: the rows of a
// wave are all read before any row of the wave is written (a cluster barrier
// between), and later waves read at or behind their own first row, which no
// earlier wave writes.  So nothing is read after it was overwritten, whatever
// the order of keep, with no scratch rows and no waiting between clusters.
//
// A copy, bound by HBM (128 requests of 4096 kept bf16 rows, 1.2 GB read and
// written: 201 us, 89 % of the copy rate; 64 requests of 1021 kept e4m3 rows 15.2,
// 73 %) or, for one request (2048 rows: 6.2), by its chain of latencies (index,
// page, row, store).  A CTA has warps that load a wave's rows into shared memory
// and warps that store them, by a bulk copy a row, and warps that look the rows
// up ahead of them; two CTAs share an SM.
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kRowsPerWave = 32;     // of a CTA
// Warps that load and that store, each an equal part of a wave's rows, and that
// look up, in turn.  A warp issues its lanes' bulk copies one after the other,
// some 70 cycles each.
constexpr int kCopyWarps = 4, kLookWarps = 4;
constexpr int kRowsPerWarp = kRowsPerWave / kCopyWarps;
constexpr int kWarpStore = kCopyWarps, kWarpLook = 2 * kCopyWarps;
constexpr int kThreads = 32 * (2 * kCopyWarps + kLookWarps);
constexpr int kLook = 8;             // waves looked up ahead
constexpr int kMaxCtas = 16;         // of a request's cluster

template <int kRowBytes>
struct CompactShape {
  static constexpr int kStages = kRowBytes > 1024 ? 3 : 6;
  static_assert(kStages < kLook, "a wave's barrier is not used again while a warp waits for it");
  static constexpr int kStageBytes = kRowsPerWave * kRowBytes;
};

struct Bars {
  uint64_t full[6], empty[6], look_full[kLook], look_empty[kLook];
  // every CTA of the cluster has its rows of the wave (of kLook waves: a storing
  // warp may be as many ahead of another as there are stages)
  uint64_t go[kLook];
  int src[kLook][kRowsPerWave], dst[kLook][kRowsPerWave];   // cache rows; dst < 0: nothing moves
  float weight[kLook][kRowsPerWave];
  int abort;
};

template <int kRowBytes>
constexpr size_t smem_bytes() {
  return CompactShape<kRowBytes>::kStages * CompactShape<kRowBytes>::kStageBytes + sizeof(Bars);
}
static_assert(kLook % kLookWarps == 0 && kRowsPerWave == 32, "a slot of looked-up rows is always the same warp's");
static_assert(2 * (smem_bytes<1152>() + 1024) <= 233472 && 2 * (smem_bytes<576>() + 1024) <= 233472, "two CTAs an SM");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}

// A bounded wait of a whole warp; false, for all of it alike, once some wait of the
// CTA has run out.
__device__ __forceinline__ bool wait(Bars* bars, const CompactArgs& a, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (__all_sync(0xffffffffu, mbar_try_wait(at, parity))) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_hint(at, parity, kWaitHintNs)) {
    if (*(volatile int*)&bars->abort) break;
    if (globaltimer() - t0 > a.wait_limit_ns) {
      *(volatile int*)&bars->abort = 1;
      if (a.status) atomicOr(a.status, 1);    // MLA_DEVERR_TIMEOUT
      break;
    }
  }
  return !__any_sync(0xffffffffu, *(volatile int*)&bars->abort);
}

template <int kRowBytes>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a, int ctas) {
  using S = CompactShape<kRowBytes>;
  constexpr int R = kRowsPerWave, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  Bars* bars = reinterpret_cast<Bars*>(smem + kStages * S::kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars->full[i]), R);
      mbar_init(smem_u32(&bars->empty[i]), kCopyWarps);
    }
    for (int i = 0; i < kLook; ++i) {
      mbar_init(smem_u32(&bars->look_full[i]), 1);
      mbar_init(smem_u32(&bars->look_empty[i]), kCopyWarps);
      mbar_init(smem_u32(&bars->go[i]), ctas);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  cluster_sync();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int len = a.keep_lens[b];
  if (len > a.max_keep) {
    if (threadIdx.x == 0 && rank == 0 && a.status) atomicOr(a.status, 2);   // MLA_DEVERR_BAD_SEQ_LEN
    len = a.max_keep;
  }
  if (len < 0) len = 0;
  const int per_wave = ctas * R;
  const int waves = (len + per_wave - 1) / per_wave;
  // the thread's row of a wave, of the CTA's R, and its row of wave w: first + w * per_wave
  const int row = warp >= kWarpLook ? lane : (warp % kCopyWarps) * kRowsPerWarp + lane;
  const int first = rank * R + row;
  float* weights = a.weights ? a.weights + (int64_t)b * a.weight_stride : nullptr;

  if (warp >= kWarpLook) {
    // ------------------------------------------------------------- look-ups
    const int32_t* keep = a.keep + (int64_t)b * a.max_keep;
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    auto index_of = [&](int w) {
      const int64_t i = first + (int64_t)w * per_wave;
      return i < len ? keep[i] : -1;
    };
    int next = index_of(warp - kWarpLook);
    for (int w = warp - kWarpLook; w < waves; w += kLookWarps) {
      const int i = first + w * per_wave, from = next;
      next = index_of(w + kLookWarps);
      const int at = w % kLook;
      int src = -1, dst = -1;
      float weight = 0.f;
      if (i < len) {
        if (from < i || from >= cap || (weights && from >= a.weight_len)) {
          if (a.status) atomicOr(a.status, 16);   // MLA_DEVERR_BAD_POSITION
        } else if (from != i) {               // else in its place already
          const int p0 = table[from / a.page_size], p1 = table[i / a.page_size];
          if (weights) weight = weights[from];
          if (p0 < 0 || p0 >= a.num_blocks || p1 < 0 || p1 >= a.num_blocks) {
            if (a.status) atomicOr(a.status, 4);  // MLA_DEVERR_BAD_BLOCK
          } else {
            src = p0 * a.page_size + from % a.page_size;
            dst = p1 * a.page_size + i % a.page_size;
          }
        }
      }
      if (!wait(bars, a, &bars->look_empty[at], ((w / kLook) & 1) ^ 1)) break;
      bars->src[at][lane] = src;
      bars->dst[at][lane] = dst;
      bars->weight[at][lane] = weight;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->look_full[at]));
    }
  } else if (warp < kWarpStore) {
    // ---------------------------------------------------------------- loads
    for (int w = 0; w < waves; ++w) {
      const int at = w % kLook, st = w % kStages;
      if (!wait(bars, a, &bars->look_full[at], (w / kLook) & 1)) break;
      if (!wait(bars, a, &bars->empty[st], ((w / kStages) & 1) ^ 1)) break;
      __syncwarp();
      const uint32_t bar = smem_u32(&bars->full[st]);
      if (lane < kRowsPerWarp) {
        if (a.debug_skip_tile && blockIdx.x == 0 && w == 0 && row == 0) {
          // test aid: the first row never comes
        } else if (bars->dst[at][row] >= 0) {
          mbar_expect_tx(bar, kRowBytes);
          bulk_load(smem_u32(smem + st * S::kStageBytes + row * kRowBytes),
                    a.cache + (int64_t)bars->src[at][row] * kRowBytes, kRowBytes, bar);
        } else {
          mbar_arrive(bar);
        }
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------------- stores
    for (int w = 0; w < waves; ++w) {
      const int at = w % kLook, st = w % kStages;
      if (!wait(bars, a, &bars->look_full[at], (w / kLook) & 1)) break;
      const int dst = lane < kRowsPerWarp ? bars->dst[at][row] : -1;
      const float weight = lane < kRowsPerWarp ? bars->weight[at][row] : 0.f;
      if (!wait(bars, a, &bars->full[st], (w / kStages) & 1)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->look_empty[at]));
      // every row of the wave is in some CTA's shared memory before one is
      // written (the arrivals order nothing but this: those rows have been read)
      if (ctas > 1) {
        if (warp == kWarpStore && lane < ctas) mbar_arrive_remote(mapa(smem_u32(&bars->go[at]), lane));
        if (!wait(bars, a, &bars->go[at], (w / kLook) & 1)) break;
        __syncwarp();
      }
      if (dst >= 0) {
        bulk_store(a.cache + (int64_t)dst * kRowBytes, smem_u32(smem + st * S::kStageBytes + row * kRowBytes), kRowBytes);
        if (weights) weights[first + w * per_wave] = weight;
      }
      bulk_commit_group();                    // one a wave, empty or not
      bulk_wait_group_read<1>();              // the wave before has left its stage
      __syncwarp();
      if (w > 0 && lane == 0) mbar_arrive(smem_u32(&bars->empty[(w - 1) % kStages]));
    }
    bulk_wait_all();
  }
  __syncwarp();
  if (*(volatile int*)&bars->abort) {
    // given up: copies in flight finish well within this time
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
  cluster_sync();                             // no CTA leaves while another may signal it
}

template <int kRowBytes>
cudaError_t launch(const CompactArgs& a, int ctas, cudaStream_t s) {
  static std::atomic<uint64_t> done{0}, wide{0};
  cudaError_t e = allow_smem(compact_kernel<kRowBytes>, smem_bytes<kRowBytes>(), done);
  if (e != cudaSuccess) return e;
  if (ctas > 8 && (e = allow_wide_clusters(compact_kernel<kRowBytes>, wide)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * (unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<kRowBytes>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, compact_kernel<kRowBytes>, a, ctas);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compact(const CompactArgs& a, int row_bytes, int sm_count, cudaStream_t s) {
  // CTAs a request: as many as its rows fill, and as are on the card at once, two
  // an SM; clusters of 16 only where they leave half of those places free (they
  // do not all find a place beside one another: 16 requests of 4096 rows 33 us
  // with 8, 35 with 16; 8 requests 22 and 19)
  int ctas = 1;
  while (ctas < kMaxCtas && (int64_t)a.batch * ctas * (ctas == 8 ? 2 : 1) <= sm_count && ctas * kRowsPerWave < a.max_keep)
    ctas *= 2;
  return row_bytes > 1024 ? launch<1152>(a, ctas, s) : launch<576>(a, ctas, s);
}

}  // namespace mla
