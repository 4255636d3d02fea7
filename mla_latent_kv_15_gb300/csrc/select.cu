// Which keys of a request stay in its cache (mla_evict_select): the first
// `sinks`, the last `recent`, and of those between them the ones of the largest
// accumulated weight, ties to the lowest index, in ascending order.
//
// A request belongs to one cluster of CTAs, each with a contiguous slice of its
// weights in shared memory.  The smallest weight kept is found by its digits:
// 32-bit codes that order as the weights do, four passes of 8 bits, a histogram
// of the digits behind the digits found so far, summed over the cluster.  Then
// every warp counts the codes above and at the threshold in its part of the
// slice, and writes its kept indices behind those of the warps before it.
//
// Bound by the passes' latency (a weight is read from memory once): barriers of
// a cluster, and the histogram's atomics, which lanes of equal digits share.
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSliceMax = 40960;     // codes of a slice held in shared memory

// Codes order as weights do: -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t code_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);     // -0 + 0 = +0
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0;   // NaN
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int ld_cluster(const int* local, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa(smem_u32(local), (uint32_t)rank)) : "memory");
  return v;
}

// kHeld: slices fit in shared memory; else codes are made from the weights in
// every pass.
template <bool kHeld>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectArgs a, int ctas) {
  extern __shared__ uint32_t codes[];
  __shared__ int hist[2][256];       // of two passes in turn: a CTA may read the last pass's beside this one's counting
  __shared__ int total[256];
  __shared__ int s_digit, s_above;
  __shared__ int s_count[2];         // codes of the slice above and at the threshold, for the cluster
  __shared__ int w_above[kWarps], w_equal[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  for (int i = tid; i < 512; i += kThreads) (&hist[0][0])[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  int n = a.seq_lens[b];
  if (n > a.weight_len) {
    if (tid == 0 && rank == 0 && a.status) atomicOr(a.status, 2);   // MLA_DEVERR_BAD_SEQ_LEN
    n = a.weight_len;
  }
  if (n < 0) n = 0;
  const int len = n < a.budget ? n : a.budget;
  int32_t* keep = a.keep + (int64_t)b * a.budget;
  const int all = ctas * kThreads, me = rank * kThreads + tid;
  for (int i = len + me; i < a.budget; i += all) keep[i] = -1;
  if (n <= a.budget) {               // every key stays
    for (int i = me; i < n; i += all) keep[i] = i;
    cluster_sync();                  // (seq_lens may be keep_lens)
    if (me == 0) a.keep_lens[b] = len;
    return;
  }
  // keys [lo, hi) compete for `need` places
  const int lo = a.sinks, hi = n - a.recent;
  const int need = a.budget - a.sinks - a.recent;
  const float* weights = a.weights + (int64_t)b * a.weight_stride;
  // every warp of the cluster has `part` keys (a multiple of 32), in order
  const int part = ((n + ctas * kWarps - 1) / (ctas * kWarps) + 31) & ~31;
  const int slice = part * kWarps;
  const int k0 = rank * slice;                          // first key of the slice
  const int beg = max(lo, k0), end = min(hi, k0 + slice);   // its competing keys
  for (int i = me; i < lo; i += all) keep[i] = i;
  for (int i = me; i < a.recent; i += all) keep[a.budget - a.recent + i] = hi + i;

  auto code_at = [&](int i) { return kHeld ? codes[i - k0] : code_of(weights[i]); };
  if (kHeld) {
    for (int i = beg + tid; i < end; i += kThreads) codes[i - k0] = code_of(weights[i]);
  }
  __syncthreads();

  // the threshold: the need-th largest code, digit by digit
  uint32_t found = 0;
  int left = need;                   // places among the codes that share the digits found
  for (int pass = 0; pass < 4 && need > 0; ++pass) {
    const int shift = 24 - 8 * pass;
    int* h = hist[pass & 1];
    for (int i0 = beg; i0 < end; i0 += kThreads) {
      const int i = i0 + tid;
      const uint32_t c = i < end ? code_at(i) : 0;
      const bool in = i < end && (pass == 0 || (c >> (shift + 8)) == found);
      // lanes of equal digits add once
      const unsigned live = __ballot_sync(0xffffffffu, in);
      if (in) {
        const int d = (c >> shift) & 255;
        const unsigned same = __match_any_sync(live, d);
        if (lane == __ffs(same) - 1) atomicAdd(&h[d], __popc(same));
      }
      __syncwarp();
    }
    cluster_sync();
    if (tid < 256) {
      int sum = 0;
      for (int r = 0; r < ctas; ++r) sum += ld_cluster(&h[tid], r);
      total[tid] = sum;
      hist[(pass & 1) ^ 1][tid] = 0;   // (every CTA has read it: before the barrier above)
    }
    __syncthreads();
    if (warp == 0) {
      // lane l has digits 255 - 8 l down to 248 - 8 l
      int own[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += own[k] = total[255 - 8 * lane - k];
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      before -= sum;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (before < left && before + own[k] >= left) {
          s_digit = 255 - 8 * lane - k;
          s_above = before;
        }
        before += own[k];
      }
    }
    __syncthreads();
    found = (found << 8) | (uint32_t)s_digit;
    left -= s_above;
  }
  // `left` of the codes equal to `found` stay, and all above it
  int above = 0, equal = 0;
  const int w0 = max(beg, k0 + warp * part), w1 = min(end, k0 + (warp + 1) * part);
  if (need > 0) {
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t c = i < w1 ? code_at(i) : 0;
      above += __popc(__ballot_sync(0xffffffffu, i < w1 && c > found));
      equal += __popc(__ballot_sync(0xffffffffu, i < w1 && c == found));
    }
  }
  if (lane == 0) {
    w_above[warp] = above;
    w_equal[warp] = equal;
  }
  __syncthreads();
  if (tid == 0) {
    int x = 0, y = 0;
    for (int w = 0; w < kWarps; ++w) {
      const int u = w_above[w], v = w_equal[w];
      w_above[w] = x;
      w_equal[w] = y;
      x += u;
      y += v;
    }
    s_count[0] = x;
    s_count[1] = y;
  }
  cluster_sync();
  if (me == 0) a.keep_lens[b] = len;
  if (need > 0 && w0 < w1) {
    above = w_above[warp];
    equal = w_equal[warp];
    for (int r = 0; r < rank; ++r) {
      above += ld_cluster(&s_count[0], r);
      equal += ld_cluster(&s_count[1], r);
    }
    const unsigned below = (1u << lane) - 1;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t c = i < w1 ? code_at(i) : 0;
      const unsigned up = __ballot_sync(0xffffffffu, i < w1 && c > found);
      const unsigned eq = __ballot_sync(0xffffffffu, i < w1 && c == found);
      const int rank_eq = equal + __popc(eq & below);
      const bool stays = (up >> lane & 1) || ((eq >> lane & 1) && rank_eq < left);
      if (stays) keep[lo + above + __popc(up & below) + min(rank_eq, left)] = i;
      above += __popc(up);
      equal += __popc(eq);
    }
  }
  cluster_sync();                    // no CTA leaves while its counts are read
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, int sm_count, cudaStream_t s) {
  // CTAs a request: a few keys a thread, all requests' on the card at once
  int ctas = 1;
  while (ctas < 8 && a.batch * ctas * 2 <= 2 * sm_count && ctas * kThreads * 4 < a.weight_len) ctas *= 2;
  const int64_t part = (((int64_t)a.weight_len + ctas * kWarps - 1) / (ctas * kWarps) + 31) / 32 * 32;
  const bool held = part * kWarps <= kSliceMax;
  const size_t smem = held ? (size_t)part * kWarps * 4 : 0;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = held ? allow_smem(select_kernel<true>, kSliceMax * 4, done) : cudaSuccess;
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch * (unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, held ? select_kernel<true> : select_kernel<false>, a, ctas);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
