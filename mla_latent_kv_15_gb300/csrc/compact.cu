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
// A copy, bound by HBM or, for one request, by how many rows its cluster has in
// flight: every thread moves one row of a wave by two bulk copies (global ->
// shared -> global), kStages waves deep, and looks its pages up two waves ahead
// (the chain keep -> block table -> row would cost a wave its time).
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

template <int kRowBytes>
struct CompactShape {
  static constexpr int kRowsPerCta = kRowBytes > 1024 ? 32 : 64;   // threads too
  static constexpr int kStages = 6;
  static constexpr int kStageBytes = kRowsPerCta * kRowBytes;
  static constexpr size_t kSmem = (size_t)kStages * (kStageBytes + kRowsPerCta * 12) + 8 * kStages;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}

template <int kRowBytes>
__global__ void __launch_bounds__(CompactShape<kRowBytes>::kRowsPerCta) compact_kernel(const CompactArgs a, int ctas) {
  using S = CompactShape<kRowBytes>;
  constexpr int R = S::kRowsPerCta, kStages = S::kStages;
  constexpr int kLead = kStages - 2;          // waves whose loads are out
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* to = reinterpret_cast<int64_t*>(smem + kStages * S::kStageBytes);   // [kStages][R] slot, -1: stays
  float* wbuf = reinterpret_cast<float*>(to + kStages * R);                    // [kStages][R]
  uint64_t* bars = reinterpret_cast<uint64_t*>(wbuf + kStages * R);
  const int t = threadIdx.x;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  if (t == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(smem_u32(&bars[i]), R);
    fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int len = a.keep_lens[b];
  if (len > a.max_keep) {
    if (t == 0 && rank == 0 && a.status) atomicOr(a.status, 2);   // MLA_DEVERR_BAD_SEQ_LEN
    len = a.max_keep;
  }
  if (len < 0) len = 0;
  const int per_wave = ctas * R;
  const int waves = (len + per_wave - 1) / per_wave;
  const int32_t* keep = a.keep + (int64_t)b * a.max_keep;
  const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
  float* weights = a.weights ? a.weights + (int64_t)b * a.weight_stride : nullptr;
  const int first = rank * R + t;

  // Two steps ahead of a wave's loads: the source index, then the two pages.
  struct Look {
    int src, pg_src, pg_dst;    // src < 0: nothing to move
    float weight;
  };
  auto index_of = [&](int w) {
    const int64_t i = (int64_t)w * per_wave + first;
    return w < waves && i < len ? keep[i] : -2;
  };
  auto pages_of = [&](int w, int src) {
    Look k{-1, 0, 0, 0.f};
    if (src == -2) return k;
    const int i = w * per_wave + first;
    const int64_t cap = (int64_t)a.max_pages * a.page_size;
    if (src < i || src >= cap || (weights && src >= a.weight_len)) {
      if (a.status) atomicOr(a.status, 16);   // MLA_DEVERR_BAD_POSITION
      return k;
    }
    if (src == i) return k;                   // in its place already
    k.src = src;
    k.pg_src = table[src / a.page_size];
    k.pg_dst = table[i / a.page_size];
    if (weights) k.weight = weights[src];
    return k;
  };
  auto issue = [&](int w, const Look& k) {
    const int st = w % kStages;
    const uint32_t bar = smem_u32(&bars[st]);
    int64_t dst = -1;
    if (k.src >= 0) {
      if (k.pg_src < 0 || k.pg_src >= a.num_blocks || k.pg_dst < 0 || k.pg_dst >= a.num_blocks) {
        if (a.status) atomicOr(a.status, 4);  // MLA_DEVERR_BAD_BLOCK
      } else {
        const int i = w * per_wave + first;
        dst = (int64_t)k.pg_dst * a.page_size + i % a.page_size;
        const int64_t src = (int64_t)k.pg_src * a.page_size + k.src % a.page_size;
        mbar_expect_tx(bar, kRowBytes);
        bulk_load(smem_u32(smem + st * S::kStageBytes + t * kRowBytes), a.cache + src * kRowBytes, kRowBytes, bar);
      }
    }
    if (dst < 0) mbar_arrive(bar);
    to[st * R + t] = dst;
    wbuf[st * R + t] = k.weight;              // (read before the wave's barrier, as the row)
  };

  int src_next = index_of(0);
  Look look = pages_of(0, src_next);
  src_next = index_of(1);
  for (int w = 0; w < kLead && w < waves; ++w) {
    const Look next = pages_of(w + 1, src_next);
    src_next = index_of(w + 2);
    issue(w, look);
    look = next;
  }
  bool dead = false;
  for (int w = 0; w < waves; ++w) {
    const int st = w % kStages, ahead = w + kLead;
    if (ahead < waves) {
      // the stage's last row has left it (this thread's own, two waves ago)
      bulk_wait_group_read<1>();
      const Look next = pages_of(ahead + 1, src_next);
      src_next = index_of(ahead + 2);
      issue(ahead, look);
      look = next;
    }
    if (!dead && !mbar_wait(smem_u32(&bars[st]), (w / kStages) & 1)) {
      dead = true;                            // nothing more is written by this thread
      if (a.status) atomicOr(a.status, 1);    // MLA_DEVERR_TIMEOUT
    }
    // every row of the wave is in some CTA's shared memory before one is written
    __syncwarp();
    cluster_sync();
    const int64_t dst = to[st * R + t];
    if (!dead && dst >= 0) {
      bulk_store(a.cache + dst * kRowBytes, smem_u32(smem + st * S::kStageBytes + t * kRowBytes), kRowBytes);
      if (weights) weights[w * per_wave + first] = wbuf[st * R + t];
    }
    bulk_commit_group();                      // one a wave, empty or not
  }
  bulk_wait_all();
}

template <int kRowBytes>
cudaError_t launch(const CompactArgs& a, int ctas, cudaStream_t s) {
  using S = CompactShape<kRowBytes>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(compact_kernel<kRowBytes>, S::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * (unsigned)ctas);
  cfg.blockDim = dim3(S::kRowsPerCta);
  cfg.dynamicSmemBytes = S::kSmem;
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
  // as many CTAs a request as give every SM one, no more than its rows fill
  const int rows = row_bytes > 1024 ? CompactShape<1152>::kRowsPerCta : CompactShape<576>::kRowsPerCta;
  int ctas = 1;
  while (ctas < 8 && a.batch * ctas * 2 <= sm_count && ctas * rows < a.max_keep) ctas *= 2;
  return row_bytes > 1024 ? launch<1152>(a, ctas, s) : launch<576>(a, ctas, s);
}

}  // namespace mla
