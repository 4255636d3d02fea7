// Work plan and join of the expanded attention.
//
// Plan: one block of threads turns the prefix sums on the device into a list
// of pieces, so that nothing of a call depends on the host knowing the lengths
// (a captured graph may be replayed over other ones).  Every sequence's query
// rows are cut into blocks of 512; a block's keys are those its last row sees;
// an item is a block and a head.  A tile of 128 keys costs two units, or one
// for a block of up to 256 rows, which the pair takes two tiles at a time.
//
// Few items (under 8 a CTA pair): all items are laid end to end, each with a
// fixed cost of kItemUnits in front (filling the pipeline, the epilogue: about
// 4000 cycles against 1300 a unit), and cut into equal spans, one a pair, so
// that every pair ends at the same time; an item on a border is cut there, in
// at most two partial pieces a pair.  (Up to 32 sequences the pairs do this by
// themselves, without this kernel.)
// Many items: the list of pieces is the same for every head, longest first,
// and the pairs take (piece, head) from it one after the other.  A block is cut
// over its keys only where it would outlast the rest: with T units over all
// heads and S pairs, a chunk is ceil(T / S), and a block of more than 1.5
// chunks is cut into ceil(cost / chunk) near-equal pieces (so the cut blocks
// of all heads number less than S and their pieces less than 2 S).
//
// The pieces' results are float32 partials with their log-sum-exp, joined by
// the combine kernel:
//   lse = ln sum_p exp(lse_p),  out = sum_p exp(lse_p - lse) out_p
// always in the order of the pieces, whichever CTAs made them.
//
// Both kernels run every instruction about once, from cold instruction
// caches, so their time is the code they fetch: loops stay loops, and what
// occurs twice is a function (the plan unrolled and inlined was 56 KB of code
// and took 8-10 us).  In a call among others the plan takes about 5 us, the join
// 4 (112 rows) to 12 (38000 rows); bound by latency both.
#include <cuda_bf16.h>

#include "prefill.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kBuckets = 1024;       // piece lengths are sorted into this many classes
constexpr int kMinChunk = kPrefillMinChunk, kItemUnits = kPrefillItemUnits;
constexpr int kMaxFixed = kPrefillFixedItems * kPrefillMaxPairs;   // blocks of a fixed plan, at most

__device__ __noinline__ int block_sum_scan(int v, int* total, int* warp_sums) {
  // exclusive scan over the block; *total: the block's sum
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    sum += warp_sums[w];
  }
  *total = sum;
  return before + incl - v;
}

using BlockOf = PrefillBlock;

// The prefix sums and the blocks before each sequence, in shared memory for
// up to kSeqs sequences (every step of a search is then a few cycles), else
// where the caller and the workspace have them.
constexpr int kSeqs = 512;
struct Sequences {
  const int *cu_q, *cu_kv, *first;
};

// Block i of the list: its sequence by binary search over the block counts.
__device__ __noinline__ BlockOf block_of(const PrefillArgs& a, const Sequences& sq_, int i) {
  int lo = 0, hi = a.batch - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sq_.first[mid] <= i) lo = mid; else hi = mid - 1;
  }
  const int q0 = sq_.cu_q[lo], sq = sq_.cu_q[lo + 1] - q0, k0 = sq_.cu_kv[lo], sk = sq_.cu_kv[lo + 1] - k0;
  return prefill_block(q0, sq, k0, sk, (i - sq_.first[lo]) * kPrefillRows, a.causal);
}

// a * b / c without overflow of the product
__device__ __noinline__ long long mul_div(long long a, int b, long long c) { return a * b / c; }

// Piece `at` of the list: key tiles [t0, t1) of a block.
__device__ __noinline__ void put_piece(const PrefillArgs& a, int at, const BlockOf& b, int t0, int t1, int prow,
                                       int head) {
  PrefillPiece r{};
  r.q0 = b.q0;
  r.nq = b.nq;
  r.kv0 = b.kv0 + t0 * kPrefillTile;
  r.nkeys = max(min(t1 * kPrefillTile, b.nkeys) - t0 * kPrefillTile, 0);
  r.lim0 = b.lim0 - t0 * kPrefillTile;
  r.prow = prow;
  r.head = head;
  if (at < a.plan.max_pieces) a.plan.pieces[at] = r;
}

// A cut block's record; returns its first partial row.
__device__ __noinline__ int put_split(const PrefillArgs& a, const BlockOf& b, int pieces, int head0, int heads,
                                      int* rows, int* splits) {
  PrefillSplit sp{};
  sp.q0 = b.q0, sp.nq = b.nq, sp.pieces = pieces, sp.head0 = head0, sp.heads = heads, sp.stride = heads * b.nq;
  sp.prow = atomicAdd(rows, pieces * heads * b.nq);
  a.plan.splits[atomicAdd(splits, 1)] = sp;
  return sp.prow;
}

__global__ void __launch_bounds__(kThreads) prefill_plan_kernel(const PrefillArgs a) {
  __shared__ int s_hist[kBuckets];
  __shared__ int s_warp[kThreads / 32];
  __shared__ int s_before[kMaxFixed];              // units of the blocks before each, fixed plan
  __shared__ int s_pair[kPrefillMaxPairs + 1];
  __shared__ long long s_border[kPrefillMaxPairs + 1];
  __shared__ int s_seq[3][kSeqs + 1];
  __shared__ BlockOf s_block[kThreads];            // few blocks: all of them
  __shared__ unsigned long long s_total;
  __shared__ int s_longest, s_status, s_rows, s_split;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (tid == 0) a.plan.header->next = 0;
  if (tid == 0) s_total = 0, s_longest = 0, s_status = 0, s_rows = 0, s_split = 0;
  __syncthreads();

  // the sequences: checks, and the blocks before each
  const bool local = a.batch <= kSeqs;
  Sequences seqs{a.cu_q, a.cu_kv, a.plan.first_block};
  int* first = a.plan.first_block;
  if (local) {
#pragma unroll 1
    for (int b = tid; b <= a.batch; b += kThreads) {
      s_seq[0][b] = a.cu_q[b];
      s_seq[1][b] = a.cu_kv[b];
    }
    seqs = Sequences{s_seq[0], s_seq[1], s_seq[2]};
    first = s_seq[2];
    __syncthreads();
  }
  int carry = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < a.batch) {
      const int q0 = seqs.cu_q[b], q1 = seqs.cu_q[b + 1], k0 = seqs.cu_kv[b], k1 = seqs.cu_kv[b + 1];
      const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_q;
      if (bad) atomicOr(&s_status, 8);
      if (k0 < 0 || k1 < k0 || k1 > a.total_kv) atomicOr(&s_status, 2);
      n = bad ? 0 : (q1 - q0 + kPrefillRows - 1) / kPrefillRows;
    }
    int total;
    const int before = block_sum_scan(n, &total, s_warp);
    if (b < a.batch) first[b] = carry + before;
    carry += total;
  }
  __syncthreads();
  const int nblocks = carry;
  if (s_status) {          // inconsistent prefix sums: flagged, nothing is computed
    if (tid == 0) {
      a.plan.header->status = s_status;
      a.plan.header->num_pieces = 0;
      a.plan.header->num_split = 0;
      a.plan.header->fixed = 0;
      a.plan.header->group_heads = 1;
    }
    return;
  }

  // a block a thread, looked up once, where there are no more
  const bool few = nblocks <= kThreads;
  auto block = [&](int i) { return few ? s_block[i] : block_of(a, seqs, i); };
  unsigned long long mine = 0;
  int longest = 0;
#pragma unroll 1
  for (int i = tid; i < nblocks; i += kThreads) {
    const BlockOf b = block_of(a, seqs, i);
    if (few) s_block[i] = b;
    mine += b.cost();
    longest = max(longest, b.cost());
  }
  if (mine) {
    atomicAdd(&s_total, mine);
    atomicMax(&s_longest, longest);
  }
  __syncthreads();
  const unsigned long long work = s_total * a.num_heads;
  longest = s_longest;

  const bool fixed = a.num_splits == 0 && longest > kMinChunk && s_total < (1ull << 30) &&
                     (long long)nblocks * a.num_heads < (long long)kPrefillFixedItems * a.pairs;
  if (fixed) {
    // fixed plan: head h's block b lies at h * all + s_before[b]
    const int items = nblocks * a.num_heads;
    int all = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < nblocks; b0 += kThreads) {
      const int b = b0 + tid;
      int total;
      const int before = block_sum_scan(b < nblocks ? block(b).cost() + kItemUnits : 0, &total, s_warp);
      if (b < nblocks) s_before[b] = all + before;
      all += total;
    }
    const long long length = (long long)all * a.num_heads;
    const int used = prefill_spans(length, items, a.pairs);
    if (tid <= kPrefillMaxPairs) {
      s_pair[tid] = 0;
      s_border[tid] = used > 0 ? mul_div(length, min(tid, used), used) : 0;   // where pair `tid`'s span begins
    }
    __syncthreads();
    int listed = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < items; i0 += kThreads) {
      const int i = i0 + tid, h = i / nblocks;
      const bool mine_is = i < items;
      BlockOf b{};
      long long s = 0;
      int p0 = 0, n = 0;
      if (mine_is) {
        b = block(i - h * nblocks);
        s = (long long)h * all + s_before[i - h * nblocks];
        int hi = used - 1;
#pragma unroll 1
        while (p0 < hi) {
          const int mid = (p0 + hi + 1) >> 1;
          if (s_border[mid] <= s) p0 = mid; else hi = mid - 1;
        }
      }
      const long long end = s + kItemUnits + b.cost();
      // two walks over the item's pieces: they are counted, then listed
      int at = 0, prow = -1;
#pragma unroll 1
      for (int walk = 0; walk < 2; ++walk) {
        if (mine_is) {
          int t0 = 0, k = 0;
#pragma unroll 1
          for (int p = p0;; ++p) {
            const long long stop = p + 1 >= used ? end : s_border[p + 1];
            const bool fin = stop >= end;
            const int t1 = fin ? b.tiles() : prefill_tiles_before(stop, s, b.unit(), b.tiles());
            if (t1 > t0 || (fin && b.tiles() == 0)) {
              if (walk) {
                put_piece(a, at + k, b, t0, t1, n > 1 ? prow + k * b.nq : -1, h);
                atomicAdd(&s_pair[p], 1);
              }
              ++k;
            }
            t0 = t1;
            if (fin) break;
          }
          n = k;
        }
        if (walk) break;
        int total;
        at = listed + block_sum_scan(n, &total, s_warp);
        listed += total;
        if (mine_is && n > 1) prow = put_split(a, b, n, h, 1, &s_rows, &s_split);
      }
    }
    __syncthreads();
    int total;
    const int count = tid < kPrefillMaxPairs ? s_pair[tid] : 0;
    const int before = block_sum_scan(count, &total, s_warp);
    if (tid <= kPrefillMaxPairs) a.plan.first_piece[tid] = before;
    carry = listed;
  } else {
    const int chunk = max((int)min((work + a.pairs - 1) / a.pairs, 1ull << 28), kMinChunk);
    const bool cut = a.num_splits == 0 && 2 * longest > 3 * chunk;
    auto pieces_of = [&](const BlockOf& b) {
      if (a.num_splits > 0) return max(1, min(a.num_splits, b.tiles()));
      return cut && 2 * b.cost() > 3 * chunk ? min((b.cost() + chunk - 1) / chunk, b.tiles()) : 1;
    };
    if (few && !cut && a.num_splits == 0) {
      // every block is a piece: its place is the number of longer ones before it
      if (tid < nblocks) {
        const BlockOf b = s_block[tid];
        int at = 0;
#pragma unroll 1
        for (int i = 0; i < nblocks; ++i) {
          const int c = s_block[i].cost();
          at += c > b.cost() || (c == b.cost() && i < tid);
        }
        put_piece(a, at, b, 0, b.tiles(), -1, 0);
      }
      carry = nblocks;
    } else {
      // length class: 0 = longest
      const int span = longest + 1;
      auto bucket = [&](int cost) { return (int)mul_div(longest - cost, kBuckets, span); };

#pragma unroll 1
      for (int i = tid; i < kBuckets; i += kThreads) s_hist[i] = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < nblocks; i += kThreads) {
        const BlockOf b = block(i);
        const int P = pieces_of(b);
#pragma unroll 1
        for (int p = 0; p < P; ++p) {
          const int t0 = (int)mul_div(b.tiles(), p, P), t1 = (int)mul_div(b.tiles(), p + 1, P);
          atomicAdd(&s_hist[bucket((t1 - t0) * b.unit())], 1);
        }
      }
      __syncthreads();
      carry = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < kBuckets; b0 += kThreads) {
        int total;
        const int v = s_hist[b0 + tid];
        const int before = block_sum_scan(v, &total, s_warp);
        s_hist[b0 + tid] = carry + before;
        carry += total;
      }
      __syncthreads();
#pragma unroll 1
      for (int i = tid; i < nblocks; i += kThreads) {
        const BlockOf b = block(i);
        const int P = pieces_of(b);
        int prow = -1;
        if (P > 1) {
          prow = put_split(a, b, P, 0, a.num_heads, &s_rows, &s_split);
        }
#pragma unroll 1
        for (int p = 0; p < P; ++p) {
          const int t0 = (int)mul_div(b.tiles(), p, P), t1 = (int)mul_div(b.tiles(), p + 1, P);
          const int at = atomicAdd(&s_hist[bucket((t1 - t0) * b.unit())], 1);
          put_piece(a, at, b, t0, t1, prow < 0 ? -1 : prow + p * a.num_heads * b.nq, 0);
        }
      }
    }
  }
  __syncthreads();
  // rows of the split blocks before each
  int rows = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < s_split; i0 += kThreads) {
    const int i = i0 + tid;
    int total;
    const int before = block_sum_scan(i < s_split ? a.plan.splits[i].nq * a.plan.splits[i].heads : 0, &total, s_warp);
    if (i < s_split) a.plan.splits[i].before = rows + before;
    rows += total;
  }
  if (tid == 0) {
    a.plan.header->split_rows = rows;
    a.plan.header->status = 0;
    a.plan.header->num_pieces = min(carry, a.plan.max_pieces);
    a.plan.header->num_split = s_split;
    a.plan.header->fixed = fixed;
    // Heads are taken in even groups whose keys and values stay in L2, but of at
    // least twice the longest item's work for every pair, which the last group's
    // long items would otherwise outlast.
    const unsigned long long least = s_total ? (2ull * longest * a.pairs + s_total - 1) / s_total : 1;
    const int group = (int)min((unsigned long long)a.num_heads, max(least, (unsigned long long)a.group_heads));
    const int groups = a.num_heads / group;
    a.plan.header->group_heads = (a.num_heads + groups - 1) / groups;
  }
}

// One warp per (row, head) of the split blocks, four output dims a lane; the
// records' row counts are searched in shared memory where they fit.
constexpr int kSearch = 1024;
static_assert(kPrefillMaxPairs <= 96, "three records a lane");

__global__ void __launch_bounds__(256) prefill_combine_kernel(const PrefillArgs a) {
  __shared__ int s_before[kSearch];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  int n = a.pairs, total;
  if (a.direct) {
    // a record a pair, most of them empty; three to a lane
    int rows[3], sum = 0;
    for (int e = 0; e < 3; ++e) {
      const int i = 3 * lane + e;
      rows[e] = i < n && a.plan.splits[i].pieces > 0 ? a.plan.splits[i].nq : 0;
      sum += rows[e];
    }
    int incl = sum;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int before = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += before;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    if (total == 0) return;
    if (threadIdx.x < 32)
      for (int e = 0, before = incl - sum; e < 3; before += rows[e], ++e) s_before[3 * lane + e] = before;
  } else {
    n = a.plan.header->num_split, total = a.plan.header->split_rows;
    if (n == 0) return;
#pragma unroll 1
    for (int i = threadIdx.x; i < n && i < kSearch; i += blockDim.x) s_before[i] = a.plan.splits[i].before;
  }
  __syncthreads();
  // the pieces behind a pair's first lie where the pairs have their first partial rows
  const int skew = a.direct ? prefill_span_rows(a.total_q) : 0;
  // consecutive rows to a warp, mostly of one record
  const int warps = gridDim.x * 8, per = (total + warps - 1) / warps;
  const int from = (blockIdx.x * 8 + (threadIdx.x >> 5)) * per, to = min(from + per, total);
  PrefillSplit sp{};
  int ends = 0;              // first row behind the record
#pragma unroll 1
  for (int rr = from; rr < to; ++rr) {
    if (rr == from || rr >= ends) {
      int lo = 0, hi = n - 1;
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int before = mid < kSearch ? s_before[mid] : a.plan.splits[mid].before;
        if (before <= rr) lo = mid; else hi = mid - 1;
      }
      sp = a.plan.splits[lo];
      if (a.direct) sp.before = s_before[lo];
      ends = sp.before + sp.nq * sp.heads;
    }
    const int own = rr - sp.before;
    const int h = own / sp.nq, r = own - h * sp.nq;
    const float* lse = a.plan.part_lse + sp.prow + own;
    const float4* part = reinterpret_cast<const float4*>(a.plan.part_o + (int64_t)(sp.prow + own) * kNope) + lane;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float ref = -INFINITY, sum = 0.f;
    // four pieces at a time; the reference follows the largest
#pragma unroll 1
    for (int p0 = 0; p0 < sp.pieces; p0 += 4) {
      float l[4];
      float4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is = p0 + e < sp.pieces;
        const int64_t at = (int64_t)(p0 + e) * sp.stride - (p0 + e > 0 ? skew : 0);
        l[e] = is ? lse[at] : -INFINITY;
        v[e] = is ? part[at * (kNope / 4)] : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      const float top = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), ref);
      const float sub = top == -INFINITY ? 0.f : top;
      const float old = expf(ref - sub);                      // ref = -inf: 0
      sum *= old, o.x *= old, o.y *= old, o.z *= old, o.w *= old;
      ref = top;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // a piece without a key has zeros; one whose weight is too small for a
        // float still counts, so that 0 * inf is NaN as in an item that is not cut
        const float w = l[e] == -INFINITY ? 0.f : expf(l[e] - sub);
        sum += w;
        o.x += w * v[e].x, o.y += w * v[e].y, o.z += w * v[e].z, o.w += w * v[e].w;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t row = (int64_t)(sp.q0 + r) * a.num_heads + sp.head0 + h;
    const __nv_bfloat162 x = __floats2bfloat162_rn(o.x * inv, o.y * inv), y = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * kNope + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : ref + logf(sum);
  }
}

cudaError_t launch_dependent(void (*kernel)(const PrefillArgs), int grid, int block, const PrefillArgs& a,
                             cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_plan(const PrefillArgs& a, cudaStream_t s) {
  return launch_dependent(prefill_plan_kernel, 1, kThreads, a, s);
}

cudaError_t launch_prefill_combine(const PrefillArgs& a, cudaStream_t s) {
  return launch_dependent(prefill_combine_kernel, 6 * a.pairs, 256, a, s);   // three blocks an SM: all run at once
}

}  // namespace mla
