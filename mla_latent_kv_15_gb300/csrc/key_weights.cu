// The attention weight of every cached key (mla_key_weights), on tcgen05:
//
//   w[j] = decay * w[j] + sum over rows (t, h) that see key j of
//          exp(scale * q[t, h] . k_j - lse[t, h])
//
// The product is taken with the keys as its rows, S = K . Q^T, so that a thread
// of the epilogue holds one key's scores and sums its exponentials along its
// own columns, with no exchange between lanes and no atomics: a key's rows are
// all summed by one CTA, in one order.
//
// CTA pairs (cta_group::2) take contiguous shares of all requests' 256-key
// tiles, 128 keys a CTA.  A tile's nine 64-column chunks stay in shared memory
// while the request's row tiles of up to 256 query rows (half of them in each
// CTA) stream past them; with one row tile a request the nine slots are a ring
// like any other.  So the cache is read once whatever the number of rows, and a
// pair's query rows once a 256-key tile.  Two accumulators of up to 256 columns
// in tensor memory (four of up to 128): a tile's exponentials run under the next
// products.
//
// An e4m3 cache is expanded to bf16 by warps of their own.  Where a request's rows
// are one tile, codes land in a ring first (kCodes: a stage of it is always the
// same one of seven warps', since loads may land out of order, and a wait two phases
// ahead would not wait).  Where they are more, shared memory is what bounds the
// kernel (see below), and eight warps take the codes from global memory into their
// registers (kDirect).  32 requests of 2048 to 16384 keys, kCodes and kDirect: 128
// rows 67 and 92 us, 192 73 and 94, 256 77 and 97, with too little on its way; 320
// rows 101 and 104, 384 121 and 107, 512 131 and 115.
//
// Measured (a launch in a graph): 64 requests of 1024 to 8192 keys, 128 heads,
// bf16 60.4 us, HBM at 90 % of the copy rate; 32 requests of 2048 to 16384 keys
// with four verified tokens (512 rows) 105 in bf16, 92 % of the tensor cores' rate,
// and 115 over e4m3 rows: there shared memory takes the expanded rows (in kCodes the
// codes too, and gives them back) and gives them to two row tiles' products beside
// the queries.  kCodes is bound by a chain: a chunk's place is free, its codes are
// widened, released to the leader, multiplied, and the place is free again once a
// tile (128 rows 67, 64 requests of 16 heads 122, where bf16 rows take 59 and 110).
// One request of 777 keys and 16 heads 7.0: a chain of loads, nine chunks' products
// and the sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                     // keys of a CTA's half of a tile (MMA rows)
constexpr int kPairKeys = 2 * kKeys;
constexpr int kChunks = kDqk / 64;             // 9
constexpr uint32_t kKBytes = kKeys * 128;      // a chunk of a CTA's keys, bf16: one 128-byte swizzled row a key
// a load of e4m3 codes: 32 keys x 192 columns, three chunks (rows of 64 bytes
// load at half the rate of rows of 128 and more)
constexpr int kRawKeys = 32, kRawChunks = 3;
constexpr uint32_t kRawRow = kRawChunks * 64, kRawBytes = kRawKeys * kRawRow;
constexpr int kRowTile = 256;                  // query rows of a product at most (its columns)
constexpr int kMaxQStages = 8;
constexpr int kWarpK = 0, kWarpQ = 1, kWarpMma = 2, kWarpEpilogue = 4, kWarpExpand = 12;
constexpr int kExpandWarps = 7;                // kCodes: each has one stage of the ring to itself
constexpr int kDirectWarps = 8;
static_assert(kDirectWarps % (kKeys / kRawKeys) == 0, "a warp always has the same 32 of a CTA's keys");
constexpr int kLseRows = 1024;                 // rows of a request whose lse is kept on chip
// e4m3: registers a thread of the issuing warps, the epilogue's and the
// expanding ones (kDirect: of both), of the launch's 96 for each of its five warpgroups
constexpr uint32_t kRegsIssue = 56, kRegsEpilogue = 112, kRegsExpand = 96, kRegsDirect = 104;
static_assert(kRegsIssue + 2 * kRegsEpilogue + 2 * kRegsExpand <= 5 * 96 && kRegsIssue + 4 * kRegsDirect <= 5 * 96,
              "register split");
constexpr float kLog2e = 1.4426950408889634f;

enum Kind { kBf16, kCodes, kDirect };   // the cache's rows; e4m3 ones by a ring of codes, or straight into registers

template <int kKind>
struct Shape {
  static constexpr int kThreads = kKind == kBf16 ? 384 : 640;
  static constexpr int kKSlots = kChunks;
  static constexpr uint32_t kQRegion = kKind == kCodes ? 32768 : 65536;   // as many stages of a CTA's half of a row tile as fit
  static constexpr int kRawStages = kKind == kCodes ? kExpandWarps : 0;
  static constexpr uint32_t kQAt = kKSlots * kKBytes;
  static constexpr uint32_t kRawAt = kQAt + kQRegion;
  static constexpr uint32_t kBarsAt = kRawAt + kRawStages * kRawBytes;
};

// Barriers marked (lead) are used in the leading CTA only, by both CTAs.
struct Bars {
  uint64_t k_full[kChunks], q_full[kMaxQStages];  // (lead) both CTAs' halves are there
  uint64_t k_empty[kChunks], q_empty[kMaxQStages];
  uint64_t raw_full[kExpandWarps], raw_empty[kExpandWarps];
  uint64_t d_full[4];
  uint64_t d_empty[4];             // (lead) the epilogue warps of both CTAs
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int tile0, tiles, b0;            // the pair's share: first tile of request b0, tiles in all
  int leads;                       // the share begins with the first tile of all
  long long sums[20];
  // lse * log2 e of the request's rows; where it has more than these, of two row
  // tiles in turn
  alignas(16) float lse2[kLseRows];
  float half[2][kKeys];            // sums of the second half of the columns
};

template <int kKind>
constexpr size_t smem_bytes() {
  return 1024 + Shape<kKind>::kBarsAt + sizeof(Bars);
}
static_assert(smem_bytes<kBf16>() <= 232448 && smem_bytes<kCodes>() <= 232448 && smem_bytes<kDirect>() <= 232448,
              "shared memory per CTA");

struct Ctx {
  Bars* bars;
  int* status;
  uint64_t limit_ns;
};

__device__ __forceinline__ void raise(const Ctx& c, int bit) {
  if (c.status) atomicOr(c.status, bit);
}

// kCluster: the acquire covers what the other CTA's threads wrote.
template <bool kCluster = false>
__device__ __forceinline__ void wait(const Ctx& c, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (kCluster ? mbar_try_wait_cluster(at, parity) : mbar_try_wait(at, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!(kCluster ? mbar_try_wait_cluster_hint(at, parity, kWaitHintNs) : mbar_try_wait_hint(at, parity, kWaitHintNs))) {
    if (*(volatile int*)&c.bars->abort) return;
    if (globaltimer() - t0 > c.limit_ns) {
      *(volatile int*)&c.bars->abort = 1;
      raise(c, 1);  // MLA_DEVERR_TIMEOUT
      return;
    }
  }
}

// Whether the CTA has given up (for the whole warp alike).  Loads and products
// stop then: a barrier that counts bytes would take an arrival too many.
__device__ __forceinline__ bool stopped(const Ctx& c) {
  return __any_sync(0xffffffffu, *(volatile int*)&c.bars->abort);
}

// A wait of a whole warp; false once the CTA has given up.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_warp(const Ctx& c, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (__all_sync(0xffffffffu, kCluster ? mbar_try_wait_cluster(at, parity) : mbar_try_wait(at, parity))) return true;
  wait<kCluster>(c, bar, parity);
  return !stopped(c);
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_once(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// 16 e4m3 codes -> 16 bf16 values (exact)
__device__ __forceinline__ void widen16(const uint4 v, uint32_t (&o)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j] & 0xFFFF), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j] >> 16), __NV_E4M3);
    const float2 flo = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 fhi = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    o[2 * j] = pack_bf16x2(flo.x, flo.y);
    o[2 * j + 1] = pack_bf16x2(fhi.x, fhi.y);
  }
}

// What a role needs of a request.
struct Request {
  int n;          // its keys
  int q0, sq;     // its query tokens
  int rows;       // sq * heads
  int row_tiles;
};

template <int kKind>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Shape<kKind>::kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                       const __grid_constant__ CUtensorMap tm_kv, const KeyWeightArgs a) {
  using S = Shape<kKind>;
  constexpr bool kFp8 = kKind != kBf16;
  constexpr int kThreads = S::kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + S::kBarsAt);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const Ctx ctx{bars, a.status, a.wait_limit_ns};
  volatile int* abort_flag = &bars->abort;

  if (tid == 0) {
    for (int i = 0; i < S::kKSlots; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), kFp8 ? 2 * kKeys / kRawKeys : 2);   // each CTA's load, or expanded loads
      mbar_init(smem_u32(&bars->k_empty[i]), 1);
    }
    for (int i = 0; i < kMaxQStages; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 2);
      mbar_init(smem_u32(&bars->q_empty[i]), 1);
    }
    for (int i = 0; i < S::kRawStages; ++i) {
      mbar_init(smem_u32(&bars->raw_full[i]), 1);
      mbar_init(smem_u32(&bars->raw_empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->d_full[i]), 1);
      mbar_init(smem_u32(&bars->d_empty[i]), 16);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_qr);
    tma_prefetch_desc(&tm_kv);
  }
  if (warp == kWarpMma) {
    tmem_alloc_pair(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish_pair();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int cap = (int)min((int64_t)a.max_pages * a.page_size, (int64_t)a.weight_len);
  auto keys_of = [&](int b) {
    const int n = a.seq_lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
  };
  // a request's query tokens, -1 where they are not within total_q; the first of them
  auto tokens_of = [&](int b, int& q0) {
    q0 = a.qsl ? a.qsl[b] : b;
    const int q1 = a.qsl ? a.qsl[b + 1] : b + 1;
    return q0 >= 0 && q0 <= q1 && q1 <= a.total_q ? q1 - q0 : -1;
  };
  auto tiles_of = [&](int b) { return b < a.batch ? (keys_of(b) + kPairKeys - 1) / kPairKeys : 0; };
  // the pair's share of all tiles: a sum over the batch, then the request that
  // holds the share's first tile
  {
    auto block_sum = [&](long long v, long long& before) {   // the block's sum, and that of the threads before this one
      long long incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      __syncthreads();
      if (lane == 31) bars->sums[warp] = incl;
      __syncthreads();
      long long all = 0;
      before = incl - v;
      for (int w = 0; w < kThreads / 32; ++w) {
        const long long u = bars->sums[w];
        before += w < warp ? u : 0;
        all += u;
      }
      return all;
    };
    const int pair = (int)cluster_id_x(), pairs = gridDim.x / 2;
    long long total = 0, before = 0;
    long long before0 = 0;                       // of the first kThreads requests, kept for the search
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      if (blockIdx.x == 0 && b < a.batch) {   // every request, those without keys too
        int q0;
        if (a.seq_lens[b] > cap) raise(ctx, 2);   // MLA_DEVERR_BAD_SEQ_LEN
        if (tokens_of(b, q0) < 0) raise(ctx, 8);  // MLA_DEVERR_BAD_QSL
      }
      total += block_sum(tiles_of(b), before);
      if (base == 0) before0 = before;
    }
    const long long lo = total * pair / pairs, hi = total * (pair + 1) / pairs;
    long long at = 0;
    for (int base = 0; base < a.batch && at <= lo; base += kThreads) {
      const int b = base + tid;
      const int tiles = tiles_of(b);
      long long all = total;
      if (a.batch <= kThreads)
        before = before0;
      else
        all = block_sum(tiles, before);
      if (at + before <= lo && lo < at + before + tiles) {
        bars->b0 = b;
        bars->tile0 = (int)(lo - at - before);
      }
      at += all;
    }
    if (tid == 0) {
      bars->tiles = (int)(hi - lo);
      bars->leads = lo == 0;
    }
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are initialised before either uses the other's
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int tiles = bars->tiles;
  const int width = a.row_tile;
  const uint32_t q_bytes = width / 2 * 128u;                   // a chunk of a CTA's half of a row tile
  const uint32_t q_stages = min(S::kQRegion / q_bytes, (uint32_t)kMaxQStages);
  const uint32_t acc_cols = width > 128 ? 256 : 128, accs = 512 / acc_cols;
  // a position in a ring, and how often it has gone round
  struct Turn {
    uint32_t at, round;
    __device__ void next(uint32_t n) {
      if (++at == n) {
        at = 0;
        ++round;
      }
    }
  };

  auto request = [&](int b) {
    Request r;
    r.n = keys_of(b);
    r.sq = max(tokens_of(b, r.q0), 0);
    r.rows = r.sq * a.num_heads;
    r.row_tiles = (r.rows + width - 1) / width;
    return r;
  };
  // calls body(request number, request, key tile) for every tile of the share
  auto for_tiles = [&](auto&& body) {
    int b = bars->b0, t = bars->tile0;
    bool fresh = true;
    Request r{};
    for (int i = 0; i < tiles; ++i, ++t) {
      while (fresh || t * kPairKeys >= r.n) {
        if (!fresh) {
          ++b;
          t = 0;
        }
        r = request(b);
        fresh = false;
      }
      body(b, r, t);
    }
  };

  auto load_keys = [&]() {
    // ------------------------------------------------------------------- keys
    uint32_t n = 0;                                // loads so far
    constexpr int kLoadKeys = kFp8 ? kRawKeys : kKeys;
    constexpr uint32_t kSlots = kFp8 ? kExpandWarps : S::kKSlots;
    const int sub_rows = a.page_size < kLoadKeys ? a.page_size : kLoadKeys;
    const int nsub = kLoadKeys / sub_rows;         // boxes of a load
    const uint64_t pol = l2_policy_evict_first();
    bool skip = a.debug_skip_tile && bars->leads && rank == 0;
    for_tiles([&](int b, const Request& r, int t) {
      if (r.row_tiles == 0) return;
      // lane l < kKeys / sub_rows: the cache row of sub-page l of the CTA's keys
      int y = (int)(a.num_blocks * a.page_size);   // past the cache: reads zeros
      const int key = t * kPairKeys + kKeys * (int)rank + lane * sub_rows;
      if (lane * sub_rows < kKeys && key < r.n) {
        const int blk = a.block_table[(int64_t)b * a.max_pages + key / a.page_size];
        if (blk >= 0 && blk < a.num_blocks)
          y = blk * a.page_size + key % a.page_size;
        else
          raise(ctx, 4);   // MLA_DEVERR_BAD_BLOCK
      }
      // e4m3: 32 keys after 32 keys of three chunks, then of the next three
      for (int c = 0; c < kChunks; c += kFp8 ? kRawChunks : 1) {
        for (int h = 0; h < kKeys / kLoadKeys; ++h, ++n) {
          const uint32_t slot = n % kSlots, round = n / kSlots;
          if (!wait_warp(ctx, kFp8 ? &bars->raw_empty[slot] : &bars->k_empty[slot], (round & 1) ^ 1)) return;
          if (skip) {      // test aid: the first load never comes
            skip = false;
            continue;
          }
          const int box = lane - h * nsub;         // the lane's box of this load
          const bool mine = box >= 0 && box < nsub;
          if constexpr (kFp8) {
            const uint32_t full = smem_u32(&bars->raw_full[slot]);
            if (lane == 0) mbar_expect_tx(full, kRawBytes);
            __syncwarp();
            if (mine)
              tma_load_2d_hint(smem_u32(smem + S::kRawAt + slot * kRawBytes) + box * sub_rows * kRawRow, &tm_kv, 64 * c,
                               y, full, pol);
          } else {
            const uint32_t full = mapa(smem_u32(&bars->k_full[slot]), 0);
            if (lane == 0) mbar_expect_tx_remote(full, kKBytes);
            __syncwarp();
            if (mine)
              tma_load_2d_pair_hint(smem_u32(smem + slot * kKBytes) + box * sub_rows * 128u, &tm_kv, 64 * c, y, full,
                                    pol);
          }
          __syncwarp();
        }
      }
    });
    // every load has landed before the CTA ends (the leader's barriers count both CTAs')
    if constexpr (kFp8) {
      for (uint32_t k = n > kSlots ? n - kSlots : 0; k < n && !*abort_flag; ++k)
        wait(ctx, &bars->raw_full[k % kSlots], (k / kSlots) & 1);
    } else if (rank == 0) {
      for (uint32_t k = n > S::kKSlots ? n - S::kKSlots : 0; k < n && !*abort_flag; ++k)
        wait(ctx, &bars->k_full[k % S::kKSlots], (k / S::kKSlots) & 1);
    }
  };
  auto load_queries = [&]() {
    // ------------------------------------------------------------- query rows
    Turn q{0, 0};
    for_tiles([&](int, const Request& r, int) {
      for (int rt = 0; rt < r.row_tiles; ++rt) {
        const int row0 = r.q0 * a.num_heads + rt * width + width / 2 * (int)rank;
        for (int c = 0; c < kChunks; ++c, q.next(q_stages)) {
          if (!wait_warp(ctx, &bars->q_empty[q.at], (q.round & 1) ^ 1)) return;
          if (elect_one()) {
            const uint32_t full = mapa(smem_u32(&bars->q_full[q.at]), 0);
            mbar_expect_tx_remote(full, q_bytes);
            tma_load_2d_pair(smem_u32(smem + S::kQAt + q.at * q_bytes), c < 8 ? &tm_q : &tm_qr, c < 8 ? 64 * c : 0, row0,
                             full);
          }
          __syncwarp();
        }
      }
    });
    if (rank == 0)
      for (uint32_t k = 0; k < q_stages && !*abort_flag; ++k, q.next(q_stages))
        if (q.round > 0) wait(ctx, &bars->q_full[q.at], (q.round - 1) & 1);   // its last load
  };
  auto multiply = [&]() {
    // --------------------------------------------------------------- products
    if (rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(256, width, 0, 0);
      constexpr uint32_t hi = desc_hi(1024, kSwizzle128B);
      const uint32_t k_lo = desc_lo(smem_u32(smem), 16), q_lo = desc_lo(smem_u32(smem + S::kQAt), 16);
      uint32_t tile = 0;                         // tiles with rows so far: each takes every key slot once
      Turn q{0, 0}, d{0, 0};
      for_tiles([&](int, const Request& r, int) {
        for (int rt = 0; rt < r.row_tiles; ++rt, d.next(accs)) {
          if (!wait_warp(ctx, &bars->d_empty[d.at], (d.round & 1) ^ 1)) return;
          for (int c = 0; c < kChunks; ++c, q.next(q_stages)) {
            if (rt == 0 && !wait_warp<kFp8>(ctx, &bars->k_full[c], tile & 1)) return;
            if (!wait_warp(ctx, &bars->q_full[q.at], q.round & 1)) return;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ka = k_lo + c * (kKBytes >> 4), qa = q_lo + q.at * (q_bytes >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_pair_ss(tmem + d.at * acc_cols, ka + 2 * k, hi, qa + 2 * k, hi, idesc, (c | k) ? 1u : 0u);
              mma_commit_pair(smem_u32(&bars->q_empty[q.at]));
              if (rt == r.row_tiles - 1) mma_commit_pair(smem_u32(&bars->k_empty[c]));
              if (c == kChunks - 1) mma_commit_pair(smem_u32(&bars->d_full[d.at]));
            }
            __syncwarp();
          }
        }
        if (r.row_tiles > 0) ++tile;
      });
      if (elect_one()) mma_commit_pair(smem_u32(&bars->drain));
      __syncwarp();
      wait(ctx, &bars->drain, 0);
    }
  };
  auto epilogue = [&]() {
    // --------------------------------------------------------------- epilogue
    const int e = tid - 32 * kWarpEpilogue;      // 0..255
    const int q4 = warp & 3, hh = e >> 7;        // tensor-memory lanes 32 q4.., 32-column groups of parity hh
    const int key = q4 * 32 + lane;
    const uint32_t from = tmem + ((uint32_t)(q4 * 32) << 16);
    Turn d{0, 0};
    uint32_t tile_no = 0, turn = 0;
    int at_b = -1;
    // lse * log2 e of one of the request's rows
    auto lse2_of = [&](const Request& r, int row) {
      const float l = a.lse[(int64_t)r.q0 * a.num_heads + row] * kLog2e;
      return l == -INFINITY ? INFINITY : l;      // a row without keys gives no weight
    };
    for_tiles([&](int b, const Request& r, int t) {
      const int j = t * kPairKeys + kKeys * (int)rank + key;
      // the first of the request's rows that sees key j (the rest follow)
      const int late = j - (r.n - r.sq);
      const int first_row = late > 0 ? late * a.num_heads : 0;
      const int first_max = __reduce_max_sync(0xffffffffu, first_row);
      const bool kept = r.rows <= kLseRows;
      if (kept && at_b != b) {
        epilogue_sync();                         // the last request's are read
        for (int row = e; row < r.rows; row += 256) bars->lse2[row] = lse2_of(r, row);
        epilogue_sync();
      }
      at_b = b;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int rt = 0; rt < r.row_tiles; ++rt, d.next(accs)) {
        const int base = rt * width, cols = min(width, r.rows - base);
        const float* lse2 = bars->lse2 + base;
        if (!kept) {
          float* to = bars->lse2 + (++turn & 1) * kRowTile;
          if (e < cols) to[e] = lse2_of(r, base + e);
          lse2 = to;
          epilogue_sync();
        }
        wait(ctx, &bars->d_full[d.at], d.round & 1);
        __syncwarp();
        tc_fence_after();
        for (int c0 = 32 * hh; c0 < cols; c0 += 64) {
          uint32_t s[32];
          tmem_ld32(from + d.at * acc_cols + c0, s);
          tmem_wait_ld();
          if (c0 + 32 <= cols && first_max <= base + c0) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lse2 + c0 + c);
              sum[0] += exp2_fast(fmaf(__uint_as_float(s[c]), a.scale_log2, -l.x));
              sum[1] += exp2_fast(fmaf(__uint_as_float(s[c + 1]), a.scale_log2, -l.y));
              sum[2] += exp2_fast(fmaf(__uint_as_float(s[c + 2]), a.scale_log2, -l.z));
              sum[3] += exp2_fast(fmaf(__uint_as_float(s[c + 3]), a.scale_log2, -l.w));
            }
          } else {
            const int lo = first_row - base - c0, hi = cols - c0;
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float p = exp2_fast(fmaf(__uint_as_float(s[c]), a.scale_log2, -lse2[c0 + c]));
              sum[c & 3] += c >= lo && c < hi ? p : 0.f;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&bars->d_empty[d.at]), 0));
      }
      const float mine = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      float* half = bars->half[tile_no++ & 1];
      if (hh == 1) half[key] = mine;
      epilogue_sync();
      if (hh == 0 && j < r.n && !*abort_flag) {
        float* w = a.weights + (int64_t)b * a.weight_stride + j;
        const float got = mine + half[key];
        *w = a.decay != 0.f ? fmaf(a.decay, *w, got) : got;
      }
    });
  };
  // 32 keys' codes of chunks c.. as bf16 into their places, 32 h of the CTA's keys on
  auto store_widened = [&](const uint4(&v)[kRawBytes / 16 / 32], int c, int h) {
    uint8_t* dst = smem + c * kKBytes + h * kRawKeys * 128;
    // 16 codes: part q of row `row`, columns 16 (q % 4) of chunk q / 4; eight rows on
    // after every three of them.  (With an address for each of the twelve the code
    // was a third longer, and 16 heads over e4m3 rows took a quarter more time.)
#pragma unroll
    for (int m = 0; m < 3; ++m) {
      const int at = lane + 32 * m, row = at / 12, q = at % 12, p = 2 * (q & 3);
      uint8_t* to = dst + (q >> 2) * kKBytes + row * 128;
      uint4* to0 = reinterpret_cast<uint4*>(to) + (p ^ (row & 7));
      uint4* to1 = reinterpret_cast<uint4*>(to) + ((p + 1) ^ (row & 7));
#pragma unroll
      for (int k = 0; k < kRawKeys / 8; ++k) {
        uint32_t o[8];
        widen16(v[3 * k + m], o);
        to0[64 * k] = make_uint4(o[0], o[1], o[2], o[3]);
        to1[64 * k] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    // the writes are in this CTA's shared memory, for the tensor cores to read,
    // before the leader hears of them: of the other CTA's by a release to the
    // cluster.  (It covers shared memory alone: one of all memory takes some 1700
    // cycles, 512 rows then 135 us instead of 115, 16 heads 158 instead of 122; by one
    // warp for all of them 124 and 140.)
    fence_proxy_async_smem();
    __syncwarp();
    if (lane < kRawChunks) {
      if (rank == 0)
        mbar_arrive(smem_u32(&bars->k_full[c + lane]));
      else
        mbar_arrive_release_smem_cluster(mapa(smem_u32(&bars->k_full[c + lane]), 0));
    }
  };
  auto expand = [&]() {
    // -------------------------------------------------------- e4m3 expansion
    const uint32_t mine = (uint32_t)(warp - kWarpExpand);   // the warp's stage
    uint32_t load = 0, tile = 0, uses = 0;                    // loads, tiles so far
    if (mine >= kExpandWarps) return;
    for_tiles([&](int, const Request& r, int) {
      if (r.row_tiles == 0) return;
      for (int c = 0; c < kChunks; c += kRawChunks) {
        for (int h = 0; h < kKeys / kRawKeys; ++h, ++load) {
          if (load % kExpandWarps != mine) continue;
          wait(ctx, &bars->raw_full[mine], uses++ & 1);
          __syncwarp();
          // the codes leave their stage at once, for its next load
          constexpr int kPieces = kRawBytes / 16 / 32;
          const uint4* src = reinterpret_cast<const uint4*>(smem + S::kRawAt + mine * kRawBytes);
          uint4 v[kPieces];
#pragma unroll
          for (int k = 0; k < kPieces; ++k) v[k] = src[lane + 32 * k];
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->raw_empty[mine]));
          // (This warp's load before this one is seven back: of the next trio of
          // chunks in the tile before, or of an earlier trio of this tile.  It
          // was written behind its own wait, and products end in order: so the
          // barriers here are at most one phase behind.)
#pragma unroll
          for (int k = 0; k < kRawChunks; ++k) wait(ctx, &bars->k_empty[c + k], (tile & 1) ^ 1);
          __syncwarp();
          store_widened(v, c, h);
        }
      }
      ++tile;
    });
  };

  auto expand_direct = [&]() {
    // -------------------------------------- e4m3 expansion from global memory
    const uint32_t mine = (uint32_t)(warp - kWarpExpand);
    const int h = (int)mine % (kKeys / kRawKeys);  // the warp's 32 of the CTA's keys
    const int shift = __ffs(a.page_size) - 1;      // (page sizes are powers of two)
    uint32_t piece = 0, tile = 0;                  // pieces of 32 keys x three chunks, and tiles, so far
    bool skip = a.debug_skip_tile && bars->leads && rank == 0;
    // the page of the lane's key of a tile, -1 behind the last; the next tile's is
    // looked up ahead
    auto page_of = [&](int b, const Request& r, int t) {
      const int key = t * kPairKeys + kKeys * (int)rank + kRawKeys * h + lane;
      return key < r.n ? a.block_table[(int64_t)b * a.max_pages + (key >> shift)] : -1;
    };
    int ahead_b = -1, ahead_t = 0, ahead = -1;
    for_tiles([&](int b, const Request& r, int t) {
      if (r.row_tiles == 0) return;
      const int key = t * kPairKeys + kKeys * (int)rank + kRawKeys * h + lane;
      const int blk = ahead_b == b && ahead_t == t ? ahead : page_of(b, r, t);
      ahead_b = b, ahead_t = t + 1, ahead = page_of(b, r, t + 1);
      int y = -1;                                  // the lane's cache row: none reads zeros
      if (key < r.n) {
        if (blk >= 0 && blk < a.num_blocks)
          y = (blk << shift) + (key & (a.page_size - 1));
        else
          raise(ctx, 4);   // MLA_DEVERR_BAD_BLOCK
      }
      for (int i = 0; i < kChunks / kRawChunks * (kKeys / kRawKeys); ++i, ++piece) {
        if (piece % kDirectWarps != mine) continue;
        if (skip) {        // test aid: the first piece never comes
          skip = false;
          continue;
        }
        const int c = i / (kKeys / kRawKeys) * kRawChunks;
        constexpr int kPieces = kRawBytes / 16 / 32;
        uint4 v[kPieces];
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          // (the places of store_widened)
          const int at = lane + 32 * m, row = at / 12;
          const uint8_t* src = a.cache + 64 * c + 16 * (at % 12);
#pragma unroll
          for (int k = 0; k < kRawKeys / 8; ++k) {
            const int from = __shfl_sync(0xffffffffu, y, row + 8 * k);
            v[3 * k + m] = make_uint4(0, 0, 0, 0);
            if (from >= 0) v[3 * k + m] = ld_once(src + (int64_t)from * kDqk);
          }
        }
        // (as above: the warp's piece before this one is eight back)
#pragma unroll
        for (int k = 0; k < kRawChunks; ++k) wait(ctx, &bars->k_empty[c + k], (tile & 1) ^ 1);
        __syncwarp();
        store_widened(v, c, h);
      }
      ++tile;
    });
  };

  if constexpr (kFp8) {
    // each warpgroup sets its register budget
    if (warp < kWarpEpilogue) {
      setmaxnreg_dec<kRegsIssue>();
      if constexpr (kKind == kCodes)
        if (warp == kWarpK) load_keys();
      if (warp == kWarpQ)
        load_queries();
      else if (warp == kWarpMma)
        multiply();
    } else if (warp < kWarpExpand) {
      setmaxnreg_inc<kKind == kDirect ? kRegsDirect : kRegsEpilogue>();
      epilogue();
    } else if constexpr (kKind == kDirect) {
      setmaxnreg_inc<kRegsDirect>();
      expand_direct();
    } else {
      setmaxnreg_dec<kRegsExpand>();
      expand();
    }
  } else {
    if (warp == kWarpK)
      load_keys();
    else if (warp == kWarpQ)
      load_queries();
    else if (warp == kWarpMma)
      multiply();
    else if (warp >= kWarpEpilogue)
      epilogue();
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
  if (warp == kWarpMma) {
    // the last signal to the peer's own barriers is on its way by now
    if (rank == 1) wait(ctx, &bars->drain, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int kKind>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_qr, const CUtensorMap& tm_kv, const KeyWeightArgs& a,
                   int sm_count, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(key_weights_kernel<kKind>, smem_bytes<kKind>(), done);
  if (e != cudaSuccess) return e;
  // no more pairs than tiles there can be
  const int64_t reach = (int64_t)a.max_pages * a.page_size < a.weight_len ? (int64_t)a.max_pages * a.page_size
                                                                          : (int64_t)a.weight_len;
  const int64_t most = a.batch * ((reach + kPairKeys - 1) / kPairKeys);
  const int pairs = sm_count / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(most < pairs ? (most > 0 ? most : 1) : pairs));
  cfg.blockDim = dim3(Shape<kKind>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<kKind>();
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, key_weights_kernel<kKind>, tm_q, tm_qr, tm_kv, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const CUtensorMap& tm_q, const CUtensorMap& tm_qr, const CUtensorMap& tm_kv, int fp8,
                               const KeyWeightArgs& a, int sm_count, cudaStream_t s) {
  // (more than one row tile a request, on average: see above)
  if (fp8 && a.many_rows) return launch<kDirect>(tm_q, tm_qr, tm_kv, a, sm_count, s);
  return fp8 ? launch<kCodes>(tm_q, tm_qr, tm_kv, a, sm_count, s) : launch<kBf16>(tm_q, tm_qr, tm_kv, a, sm_count, s);
}

}  // namespace mla
