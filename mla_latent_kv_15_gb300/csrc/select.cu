// Which keys of a request stay in its cache (mla_evict_select): the first
// `sinks`, the last `recent`, and of those between them the ones of the largest
// accumulated weight, ties to the lowest index, in ascending order.
//
// A request belongs to one cluster of CTAs, each with a contiguous slice of its
// weights in shared memory, as 32-bit codes that order as the weights do.  The
// smallest code kept is found by its digits, 11, 11 and 10 bits from the top: a
// histogram of the digit behind the digits found so far, summed over the
// cluster, gives the digit that holds the last place.  (Weights are positive,
// so the first digit is the exponent and two bits of the mantissa: few codes
// are left for the second.)  Then every warp counts the codes above and at the
// threshold in its part of the slice, and writes its kept indices behind those
// of the warps before it.
//
// A weight is read from memory once.  128 requests of 8192 to 32768 keys take 13.4
// us where the weights' bytes need 1.8: a chain of passes in one CTA a request, on
// 128 of 152 SMs, and as much the passes' instructions (58 % of the issue slots, 4.9
// M warp instructions for 1.05 M keys; the longest request is the time of all).  The
// last of them has its codes and the first histogram after 3.7, the three digits after 4.3,
// 6.7 and 8.1, its votes after 10.8 and its indices after 12.6; one request of 4096
// keys (7.1) 1.9, 2.5, 3.5, 4.2, 5.0 and 6.2.  Eight loads of four weights are in
// flight a thread; the kept keys come from votes that a lane holds for 32 keys, so
// that the codes are not read twice more (16.5 without).
#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kSliceMax = 40960;     // codes of a slice held in shared memory

// Codes order as weights do: -0 as +0, NaN below everything.  0 is no weight's
// code: that of the keys which do not compete.
__device__ __forceinline__ uint32_t code_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);     // -0 + 0 = +0
  const uint32_t c = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return w == w ? c : 1;                           // (-infinity's is 0x007fffff)
}

__device__ __forceinline__ int ld_cluster(const int* local, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa(smem_u32(local), (uint32_t)rank)) : "memory");
  return v;
}
__device__ __forceinline__ int2 ld_cluster2(const int* local, int rank) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(mapa(smem_u32(local), (uint32_t)rank))
               : "memory");
  return v;
}

__device__ __forceinline__ int warp_incl_scan(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

struct Shared {
  alignas(16) int hist[2][kBins];    // of two digits in turn: one is read by the cluster while the other is counted
  int warp_sum[kWarps];
  int digit, above;
  int count[2];                      // codes of the slice above and at the threshold, for the cluster
  int w_above[kWarps], w_equal[kWarps];
};

// kHeld: slices fit in shared memory; else codes are made from the weights in
// every pass.
template <bool kHeld>
__global__ void __launch_bounds__(kThreads, 1) select_kernel(const SelectArgs a, int ctas) {
  extern __shared__ __align__(16) uint32_t codes[];
  __shared__ Shared sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  auto cluster_wide = [&]() {
    if (ctas > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  for (int i = tid; i < kBins; i += kThreads) sm.hist[0][i] = 0;
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
    cluster_wide();                  // (seq_lens may be keep_lens)
    if (me == 0) a.keep_lens[b] = len;
    return;
  }
  // Keys are counted from the 16-byte boundary before the row's weights, `shift`
  // weights ahead of the first, so that four at a time can be loaded.
  const float* weights = a.weights + (int64_t)b * a.weight_stride;
  const int shift = (int)(reinterpret_cast<uintptr_t>(weights) / 4 % 4);
  // keys [lo, hi) compete for `need` places
  const int lo = a.sinks, hi = n - a.recent;
  const int need = a.budget - a.sinks - a.recent;
  // every warp of the cluster has `part` of them (a multiple of 128), in order
  const int part = ((n + 3 + ctas * kWarps - 1) / (ctas * kWarps) + 127) & ~127;
  const int slice = part * kWarps;
  const int k0 = rank * slice;                              // first of the slice
  const int beg = max(lo + shift - k0, 0), end = min(hi + shift - k0, slice);   // its competing keys, from k0
  const float* own = weights - shift + k0;
  const int held = (end + 3) & ~3;                          // codes looked at, four a thread and step
  __syncthreads();

  if (need > 0) {
    // the codes, and the first digit's histogram: kAtOnce quads of a thread in
    // flight.  (Code 0 is counted too: it is below every place.)
    constexpr int kAtOnce = 8;
    for (int base = 4 * tid; base < held; base += 4 * kAtOnce * kThreads) {
      float4 w[kAtOnce];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = base + 4 * k * kThreads;
        if (i >= beg && i + 4 <= end)
          w[k] = *reinterpret_cast<const float4*>(own + i);
        else
          w[k] = make_float4(i >= beg && i < end ? own[i] : 0.f, i + 1 >= beg && i + 1 < end ? own[i + 1] : 0.f,
                             i + 2 >= beg && i + 2 < end ? own[i + 2] : 0.f, i + 3 >= beg && i + 3 < end ? own[i + 3] : 0.f);
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int i = base + 4 * k * kThreads;
        if (i >= held) break;
        uint32_t c[4] = {code_of(w[k].x), code_of(w[k].y), code_of(w[k].z), code_of(w[k].w)};
        if (i < beg || i + 4 > end) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < beg || i + e >= end) c[e] = 0;
        }
        if (kHeld) *reinterpret_cast<uint4*>(codes + i) = make_uint4(c[0], c[1], c[2], c[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) atomicAdd(&sm.hist[0][c[e] >> 21], 1);
      }
    }
    __syncthreads();
  }
  auto codes_at = [&](int i0, uint32_t (&c)[4]) {
    if (kHeld) {
      const uint4 v = *reinterpret_cast<const uint4*>(codes + i0);
      c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = i0 + k >= beg && i0 + k < end ? code_of(own[i0 + k]) : 0;
    }
  };

  // the threshold: the need-th largest code, digit by digit
  uint32_t found = 0;
  int left = need;                   // places among the codes that share the digits found
  for (int pass = 0; pass < 3 && need > 0; ++pass) {
    int* h = sm.hist[pass & 1];
    if (pass > 0) {
      const int shift = pass == 1 ? 10 : 0, above = pass == 1 ? 21 : 10;
      const uint32_t mask = pass == 1 ? 2047 : 1023;
      for (int i0 = 4 * tid; i0 < held; i0 += 4 * kThreads) {
        uint32_t c[4];
        codes_at(i0, c);
        bool any = false;            // (few codes share the digits found)
#pragma unroll
        for (int k = 0; k < 4; ++k) any |= (c[k] >> above) == found;
        if (any) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((c[k] >> above) == found) atomicAdd(&h[c[k] >> shift & mask], 1);
        }
      }
    }
    cluster_wide();
    // thread t has bins kBins - 2 t - 2 and kBins - 2 t - 1: from the top down
    const int top = kBins - 2 * (tid + 1);
    int2 v = make_int2(0, 0);
    for (int r = 0; r < ctas; ++r) {
      const int2 u = ctas > 1 ? ld_cluster2(h + top, r) : *reinterpret_cast<const int2*>(h + top);
      v.x += u.x, v.y += u.y;
    }
    // (the other histogram was read by every CTA before the barrier above)
    *reinterpret_cast<int2*>(sm.hist[(pass & 1) ^ 1] + top) = make_int2(0, 0);
    const int sum = v.x + v.y;
    const int incl = warp_incl_scan(sum);
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    const int sums = sm.warp_sum[lane];      // of warp `lane`
    const int before = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0);
    if (before < left && before + sum >= left) {
      const bool upper = before + v.y >= left;
      sm.digit = upper ? top + 1 : top;
      sm.above = upper ? before : before + v.y;
    }
    __syncthreads();
    found = pass == 2 ? (found << 10) | (uint32_t)sm.digit : (found << 11) | (uint32_t)sm.digit;
    left -= sm.above;
  }
  // `left` of the codes equal to `found` stay, and all above it.  Of 1024 keys of
  // a warp, a lane holds the votes on 32: which are above, which at the threshold.
  const int w0 = warp * part, w1 = min(held, w0 + part);     // the warp's keys, counted from k0
  uint2* words = reinterpret_cast<uint2*>(codes + slice);    // kHeld: [slice / 32]
  auto vote = [&](int g0) {
    uint2 mine = make_uint2(0, 0);
    const int rows = min((w1 - g0 + 31) / 32, 32);
#pragma unroll 4
    for (int k = 0; k < rows; ++k) {
      const int i = g0 + 32 * k + lane;
      uint32_t c = 0;
      if (i < w1) c = kHeld ? codes[i] : (i >= beg && i < end ? code_of(own[i]) : 0);
      const unsigned up = __ballot_sync(0xffffffffu, c > found), eq = __ballot_sync(0xffffffffu, c == found);
      if (lane == k) mine = make_uint2(up, eq);
    }
    return mine;
  };
  int above = 0, equal = 0;
  if (need > 0) {
    for (int g0 = w0; g0 < w1; g0 += 1024) {
      const uint2 v = vote(g0);
      if (kHeld && g0 + 32 * lane < w0 + part) words[g0 / 32 + lane] = v;
      above += __popc(v.x);
      equal += __popc(v.y);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
  }
  if (lane == 0) {
    sm.w_above[warp] = above;
    sm.w_equal[warp] = equal;
  }
  __syncthreads();
  const int of_above = sm.w_above[lane], of_equal = sm.w_equal[lane];   // of warp `lane`
  const int sum_above = __reduce_add_sync(0xffffffffu, of_above);
  const int sum_equal = __reduce_add_sync(0xffffffffu, of_equal);
  above = __reduce_add_sync(0xffffffffu, lane < warp ? of_above : 0);
  equal = __reduce_add_sync(0xffffffffu, lane < warp ? of_equal : 0);
  if (tid == 0) {
    sm.count[0] = sum_above;
    sm.count[1] = sum_equal;
  }
  cluster_wide();
  if (me == 0) a.keep_lens[b] = len;
  for (int i = me; i < lo; i += all) keep[i] = i;
  for (int i = me; i < a.recent; i += all) keep[a.budget - a.recent + i] = hi + i;
  if (need > 0 && w0 < w1) {
    for (int r = 0; r < rank; ++r) {
      above += ld_cluster(&sm.count[0], r);
      equal += ld_cluster(&sm.count[1], r);
    }
    const int key0 = k0 - shift;
    for (int g0 = w0; g0 < w1; g0 += 1024) {
      uint2 v = make_uint2(0, 0);
      if (!kHeld)
        v = vote(g0);
      else if (g0 + 32 * lane < w0 + part)
        v = words[g0 / 32 + lane];
      // of the lane's keys at the threshold, as many as there are places
      const int eqs = __popc(v.y), eq_incl = warp_incl_scan(eqs);
      int places = left - (equal + eq_incl - eqs);
      uint32_t stay = v.x;
      for (uint32_t e = v.y; e && places > 0; e &= e - 1, --places) stay |= e & (0u - e);
      const int ups = __popc(v.x), up_incl = warp_incl_scan(ups);
      int at = lo + above + up_incl - ups + min(equal + eq_incl - eqs, left);
      for (; stay; stay &= stay - 1) keep[at++] = key0 + g0 + 32 * lane + __ffs(stay) - 1;
      above += __shfl_sync(0xffffffffu, up_incl, 31);
      equal += __shfl_sync(0xffffffffu, eq_incl, 31);
    }
  }
  if (ctas > 1) cluster_sync();      // no CTA leaves while its counts are read
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, int sm_count, cudaStream_t s) {
  // CTAs a request: a few keys a thread, all requests' on the card at once.  Both
  // this and whether codes are held go by the rows' width, the most keys a request
  // can have, since the lengths are the device's: rows far wider than their requests
  // are long cost 7 us (one request of 4096 keys 7.1, in rows of 40960 14.6; 128 of
  // 8192 to 32768 13.6, in rows of 40960 or 131072 21.1)
  int ctas = 1;
  while (ctas < 8 && (int64_t)a.batch * ctas * 2 <= sm_count && ctas * kThreads * 8 < a.weight_len) ctas *= 2;
  const int64_t part = (((int64_t)a.weight_len + 3 + ctas * kWarps - 1) / (ctas * kWarps) + 127) / 128 * 128;
  const bool held = part * kWarps <= kSliceMax;
  const size_t smem = held ? (size_t)part * kWarps * 4 + part * kWarps / 32 * 8 : 0;   // the codes, and the votes on them
  static std::atomic<uint64_t> done{0};
  cudaError_t e = held ? allow_smem(select_kernel<true>, kSliceMax * 4 + kSliceMax / 4, done) : cudaSuccess;
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
