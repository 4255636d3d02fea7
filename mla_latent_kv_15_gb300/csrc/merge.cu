// LSE merge kernels (merge_attn_states of the MLA pages: combine partial
// attention results over disjoint key sets by their log-sum-exp).
//
//  * combine_kernel: after a split-KV decode, merges the k partials of every
//    split group (fp16 codes with a power-of-two scale per 32-dim chunk, fp32
//    LSE) into the final bf16 output and LSE, and zero-fills groups that see
//    no key (o = 0, lse = -inf).
//  * merge2_kernel: the public two-way merge (mla_merge_states).
//
// Both stream with 16-byte vector loads over a grid sized in multiples of the
// SM count (of the current device, queried by the caller on every call).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace mla {
namespace {

// acc[0..7] += w * the eight fp16 codes in v (a partial's codes times w x its scale)
__device__ __forceinline__ void accumulate(float* acc, float w, const uint4 v) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(h[k]);
    acc[2 * k] = fmaf(w, f.x, acc[2 * k]);
    acc[2 * k + 1] = fmaf(w, f.y, acc[2 * k + 1]);
  }
}

// Merge of the split groups' partials.  The work item is (group, rows
// 4y..4y+3); 64 threads take an item, 16 per row and 32 dims per thread
// (dims 128c + 8s .. 128c + 8s + 7 for c = 0..3 of thread s, so that every
// load instruction of a warp reads whole 256-byte runs), and a block of 256
// threads holds four items at once.
// The kernel is bound by the latency of its loads: every load of an item's
// pieces is issued before any use, and the next item's group record loads
// while the current one merges.  One wave of blocks (as many as are
// resident on every SM at once) strides over the items.
__global__ void __launch_bounds__(256, 2) combine_kernel(const DecodeArgs a) {
  const Plan& P = a.plan;
  constexpr int kQuads = kRows / 4;   // items per group
  // pieces whose loads are all in flight at once: with the balanced split a
  // group spans at most three CTA-pair spans unless it is longer than two
  constexpr int kFew = 3;
  constexpr int kChunks = kLkv / 32;  // scales per partial row
  const int VG = (int)gridDim.x * 4;  // item slots of the grid
  const int cap = P.max_groups * kQuads;
  // The plan's records are complete before this grid starts: the decode
  // kernel lets it launch only after its own wait for the plan grid.  So the
  // header and the first record are read before the wait for the decode
  // grid, which only the partials need.
  int item = (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6);
  GroupRec gnext{};
  if (item < cap) gnext = P.groups[item / kQuads];
  const int items = min(cap, P.header->num_groups * kQuads);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the next kernel on the stream may launch (it waits for this grid)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);
  const int sub = threadIdx.x & 15;              // dims 128 c + 8 sub .. + 7, c = 0..3
  const int d0 = sub * 8;
  const int quad_row = (threadIdx.x >> 4) & 3;   // row of the item
  for (; item < items; item += VG) {
    const GroupRec gr = gnext;
    if (item + VG < items) gnext = P.groups[(item + VG) / kQuads];
    if (gr.pieces == 1) continue;  // written directly by the decode kernel
    const int r = (item % kQuads) * 4 + quad_row;
    if (r >= gr.nrows || gr.row0 + r >= a.total_rows) continue;
    const int R = gr.row0 + r;
    float acc[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) acc[k] = 0.f;
    float lse = -INFINITY;
    if (gr.pieces <= kFew) {
      // the usual case: every load of every piece issued before any use
      float l[kFew], sc[kFew][4];
      uint4 x[kFew][4];
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        l[i] = -INFINITY;
        if (i < gr.pieces) {
          const size_t at = (size_t)(gr.ubase + i) * kRows + r;
          l[i] = P.part_lse[at];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sc[i][c] = P.part_scale[at * kChunks + 4 * c + (sub >> 2)];
            x[i][c] = *reinterpret_cast<const uint4*>(P.part_o + at * kLkv + 128 * c + d0);
          }
        }
      }
      float mx = l[0];
#pragma unroll
      for (int i = 1; i < kFew; ++i) mx = fmaxf(mx, l[i]);
      if (mx != -INFINITY) {
        float wsum = 0.f;
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
          if (i < gr.pieces) {
            const float w = __expf(l[i] - mx);
            wsum += w;
#pragma unroll
            for (int c = 0; c < 4; ++c) accumulate(acc + 8 * c, w * sc[i][c], x[i][c]);
          }
        }
        const float inv = 1.f / wsum;
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] *= inv;
        lse = mx + __logf(wsum);
      }
    } else {
      // more pieces than registers (num_splits > kFew): one piece at a time
      float mx = -INFINITY;
      for (int i = 0; i < gr.pieces; ++i) mx = fmaxf(mx, P.part_lse[(size_t)(gr.ubase + i) * kRows + r]);
      if (mx != -INFINITY) {
        float wsum = 0.f;
        for (int i = 0; i < gr.pieces; ++i) {
          const size_t at = (size_t)(gr.ubase + i) * kRows + r;
          const float w = __expf(P.part_lse[at] - mx);
          wsum += w;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            accumulate(acc + 8 * c, w * P.part_scale[at * kChunks + 4 * c + (sub >> 2)],
                       *reinterpret_cast<const uint4*>(P.part_o + at * kLkv + 128 * c + d0));
        }
        const float inv = 1.f / wsum;
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] *= inv;
        lse = mx + __logf(wsum);
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint4 v;
      __nv_bfloat162 h;
      h = __floats2bfloat162_rn(acc[8 * c + 0], acc[8 * c + 1]); v.x = *reinterpret_cast<uint32_t*>(&h);
      h = __floats2bfloat162_rn(acc[8 * c + 2], acc[8 * c + 3]); v.y = *reinterpret_cast<uint32_t*>(&h);
      h = __floats2bfloat162_rn(acc[8 * c + 4], acc[8 * c + 5]); v.z = *reinterpret_cast<uint32_t*>(&h);
      h = __floats2bfloat162_rn(acc[8 * c + 6], acc[8 * c + 7]); v.w = *reinterpret_cast<uint32_t*>(&h);
      *reinterpret_cast<uint4*>(out + (size_t)R * kLkv + 128 * c + d0) = v;
    }
    if (a.lse && sub == 0) a.lse[R] = lse;
  }
}

// The merge of mla_decode_shared: a row's partials are those of its own keys and
// those of the row among its prefix's, as the plan's records say; a prefix cut
// over many pairs leaves up to one a pair.  64 threads a row, eight dims each,
// and so few registers a partial that the loads of kMany are in flight at once.
// A block joins four rows at a time or, where no more rows than blocks are, one
// row whose partials its four parts share.  (With 16 threads a row and four
// partials at once the join of 64 rows over ten partials took 7.7 us, now 1.6;
// 8192 rows of 512 over two or three take 10, 60 % of the copy rate.  Four blocks
// an SM with four partials at once: many prefixes 36.8 -> 32.5, but batches of few
// rows 1 to 3.6 us slower.)  Rows
// that the decode wrote itself (one piece, and no prefix keys) are left.
struct Joined {
  float mx, wsum, acc[8];
};

__global__ void __launch_bounds__(256, 2) combine_shared_kernel(const DecodeArgs a) {
  const Plan& P = a.plan;
  constexpr int kMany = 8;
  __shared__ Joined s_part[3][64];
  const PlanHeader head = *P.header;
  const bool single = (long long)(head.num_groups - head.own_groups) * head.own_rows <= gridDim.x;
  const int per = single ? 1 : 4;              // rows of an item
  const int row_items = (head.own_rows + per - 1) / per;   // of a group: as many as the largest has
  const int items = head.num_groups * row_items;
  int item = head.own_groups * row_items + (int)blockIdx.x;
  // (the plan is complete before this grid starts: the first record is read
  // before the wait for the partials)
  JoinRec next{};
  if (item < items) next = P.joins[item / row_items];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out);
  const int sub = threadIdx.x & 63, part = threadIdx.x >> 6;
  const int first = single ? part : 0, step = single ? 4 : 1;   // the thread's partials of its row
  for (; item < items; item += (int)gridDim.x) {
    const JoinRec gr = next;
    if (item + (int)gridDim.x < items) next = P.joins[(item + (int)gridDim.x) / row_items];
    const int r = (item % row_items) * per + (single ? 0 : part);
    if (r >= gr.nrows || gr.row0 + r >= a.total_rows) continue;   // (the whole block where it shares a row)
    const bool second = r >= gr.split;
    const int pre = second ? gr.pre2_pieces : gr.pre_pieces;
    const int n = gr.own_pieces + pre;
    if (pre == 0 && gr.own_pieces == 1) continue;   // written by the decode kernel
    const size_t pre_at = second ? gr.pre2_at + (r - gr.split) : gr.pre_at + r, own_at = gr.own_at + r;
    Joined j{-INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}};
    // kMany partials at a time, each merged into what those before left
    for (int i0 = first; i0 < n; i0 += kMany * step) {
      float l[kMany], sc[kMany];
      uint4 x[kMany];
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        const int k = i0 + i * step;
        l[i] = -INFINITY;
        if (k < n) {
          const size_t p = k < pre ? pre_at + (size_t)k * kRows : own_at + (size_t)(k - pre) * kRows;
          l[i] = P.part_lse[p];
          sc[i] = P.part_scale[p * (kLkv / 32) + (sub >> 2)];
          x[i] = *reinterpret_cast<const uint4*>(P.part_o + p * kLkv + 8 * sub);
        }
      }
      float top = j.mx;
#pragma unroll
      for (int i = 0; i < kMany; ++i) top = fmaxf(top, l[i]);
      if (top == -INFINITY) continue;
      const float keep = __expf(j.mx - top);
      j.wsum *= keep;
#pragma unroll
      for (int k = 0; k < 8; ++k) j.acc[k] *= keep;
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        if (i0 + i * step < n) {
          const float w = __expf(l[i] - top);
          j.wsum += w;
          accumulate(j.acc, w * sc[i], x[i]);
        }
      }
      j.mx = top;
    }
    if (single) {
      // the four parts, in their order
      __syncthreads();
      if (part > 0) s_part[part - 1][sub] = j;
      __syncthreads();
      if (part > 0) continue;
      float top = j.mx;
#pragma unroll
      for (int i = 0; i < 3; ++i) top = fmaxf(top, s_part[i][sub].mx);
      if (top != -INFINITY) {
        const float keep = __expf(j.mx - top);
        j.wsum *= keep;
#pragma unroll
        for (int k = 0; k < 8; ++k) j.acc[k] *= keep;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const Joined& o = s_part[i][sub];
          const float w = __expf(o.mx - top);
          j.wsum += w * o.wsum;
#pragma unroll
          for (int k = 0; k < 8; ++k) j.acc[k] = fmaf(w, o.acc[k], j.acc[k]);
        }
        j.mx = top;
      }
    }
    float lse = -INFINITY;
    if (j.mx != -INFINITY) {
      const float inv = 1.f / j.wsum;
#pragma unroll
      for (int k = 0; k < 8; ++k) j.acc[k] *= inv;
      lse = j.mx + __logf(j.wsum);
    }
    uint4 v;
    __nv_bfloat162 h;
    h = __floats2bfloat162_rn(j.acc[0], j.acc[1]); v.x = *reinterpret_cast<uint32_t*>(&h);
    h = __floats2bfloat162_rn(j.acc[2], j.acc[3]); v.y = *reinterpret_cast<uint32_t*>(&h);
    h = __floats2bfloat162_rn(j.acc[4], j.acc[5]); v.z = *reinterpret_cast<uint32_t*>(&h);
    h = __floats2bfloat162_rn(j.acc[6], j.acc[7]); v.w = *reinterpret_cast<uint32_t*>(&h);
    const size_t R = (size_t)(gr.row0 + r);
    *reinterpret_cast<uint4*>(out + R * kLkv + 8 * sub) = v;
    if (a.lse && sub == 0) a.lse[R] = lse;
  }
}

template <bool kBf16>
__device__ __forceinline__ void load8(const void* base, size_t idx, float (&x)[8]) {
  if (kBf16) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + idx);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __bfloat1622float2(h[k]);
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
    const float4 a = p[0], b = p[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

template <bool kBf16>
__device__ __forceinline__ void store8(void* base, size_t idx, const float (&x)[8]) {
  if (kBf16) {
    uint4 v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + idx) = v;
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + idx);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// One thread per 8 consecutive elements of a row; grid-stride over all vectors.
template <bool kBf16>
__global__ void __launch_bounds__(256) merge2_kernel(const void* __restrict__ o_a, const float* __restrict__ lse_a,
                                                     const void* __restrict__ o_b, const float* __restrict__ lse_b,
                                                     int64_t rows, int dim, void* out, float* lse_out) {
  const int vpr = dim / 8;
  const int64_t nvec = rows * vpr;
  for (int64_t v = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; v < nvec; v += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = v / vpr;
    const size_t idx = (size_t)r * dim + (size_t)(v - r * vpr) * 8;
    const float la = lse_a[r], lb = lse_b[r];
    const float mx = fmaxf(la, lb);
    float x[8], y[8];
    load8<kBf16>(o_a, idx, x);
    load8<kBf16>(o_b, idx, y);
    float res[8];
    float lse;
    if (mx == -INFINITY) {
#pragma unroll
      for (int k = 0; k < 8; ++k) res[k] = 0.f;
      lse = -INFINITY;
    } else {
      const float wa = __expf(la - mx), wb = __expf(lb - mx);
      const float inv = 1.f / (wa + wb);
#pragma unroll
      for (int k = 0; k < 8; ++k) res[k] = (wa * x[k] + wb * y[k]) * inv;
      lse = mx + __logf(wa + wb);
    }
    store8<kBf16>(out, idx, res);
    if (lse_out && v - r * vpr == 0) lse_out[r] = lse;
  }
}

}  // namespace

cudaError_t launch_combine(const DecodeArgs& a, int max_groups, int sm_count, cudaStream_t s) {
  // one wave: as many blocks as are resident on every SM at once (a block
  // beyond that would start only when another ends), or fewer when the plan
  // cannot hold as many items
  static const int per_sm = [] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, combine_kernel, 256, 0) != cudaSuccess || n < 1) n = 1;
    return n;
  }();
  cudaLaunchConfig_t cfg = {};
  const long long max_items = (long long)max_groups * (kRows / 4);
  long long blocks = (long long)(sm_count > 0 ? sm_count : 1) * per_sm;
  if (blocks * 4 > max_items) blocks = (max_items + 3) / 4;   // four items per block at once
  if (blocks < 1) blocks = 1;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, combine_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_combine_shared(const DecodeArgs& a, int sm_count, cudaStream_t s) {
  const long long max_rows = a.total_rows;
  long long blocks = (long long)(sm_count > 0 ? sm_count : 1) * 2;
  if (blocks > max_rows) blocks = max_rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < 1 ? 1 : blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, combine_shared_kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_merge_states(const void* o_a, const float* lse_a, const void* o_b, const float* lse_b,
                                int64_t rows, int dim, int o_is_bf16, void* out, float* lse_out, int sm_count,
                                cudaStream_t s) {
  const int64_t nvec = rows * (dim / 8);
  int64_t blocks = (nvec + 255) / 256;
  const int64_t cap = (int64_t)(sm_count > 0 ? sm_count : 1) * 8;
  if (blocks > cap) blocks = cap;
  if (blocks < 1) blocks = 1;
  if (o_is_bf16)
    merge2_kernel<true><<<(unsigned)blocks, 256, 0, s>>>(o_a, lse_a, o_b, lse_b, rows, dim, out, lse_out);
  else
    merge2_kernel<false><<<(unsigned)blocks, 256, 0, s>>>(o_a, lse_a, o_b, lse_b, rows, dim, out, lse_out);
  return cudaGetLastError();
}

}  // namespace mla
