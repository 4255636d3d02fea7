// The attention weight of every cached key (mla_key_weights), on tcgen05:
//
//   w[j] = decay * w[j] + sum over rows (t, h) that see key j of
//          exp(scale * q[t, h] . k_j - lse[t, h])
//
// The product is taken with the keys as its rows, S = K . Q^T: 128 keys by up
// to 128 query rows, so that a thread of the epilogue holds one key's scores
// and sums its exponentials along its own columns, with no exchange between
// lanes and no atomics: a key's rows are all summed by one CTA, in one order.
//
// A CTA takes a contiguous share of all requests' 128-key tiles, and for each
// the request's row tiles in turn; both operands stream through a ring in
// 64-column chunks (one 128-byte swizzled row a key or query row).  An e4m3
// cache lands as codes beside the chunk and is expanded to bf16 by four warps.
// Two accumulators in tensor memory: a tile's exponentials run under the next
// one's products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                     // keys of a tile (MMA M)
constexpr int kChunks = kDqk / 64;             // 9
constexpr uint32_t kKBytes = kKeys * 128;      // a chunk of a key tile, bf16
constexpr uint32_t kRawBytes = kKeys * 64;     // the same as e4m3 codes
constexpr uint32_t kQBytes = 128 * 128;        // a chunk of up to 128 query rows
constexpr int kThreads = 512;                  // warp 0 loads, 1 issues, 4-11 epilogue, 12-15 expand e4m3
constexpr int kWarpEpilogue = 4, kWarpExpand = 12;
constexpr float kLog2e = 1.4426950408889634f;

template <bool kFp8>
struct Shape {
  static constexpr uint32_t kStage = kKBytes + kQBytes + (kFp8 ? kRawBytes : 0);
  static constexpr int kStages = kFp8 ? 5 : 6;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + 4096;
};

struct Bars {
  uint64_t full[6], empty[6], raw_full[6];
  uint64_t d_full[2], d_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int tile0, tiles, b0;           // this CTA's share: first tile of request b0, tiles in all
  int leads;                      // the share begins with the first tile of all
  long long sums[kThreads / 32];
  float lse2[2][128];             // lse * log2 e of the row tile's rows, two tiles in turn
  float half[2][kKeys];           // sums of the second column half
};
static_assert(sizeof(Bars) <= 4096, "fits behind the stages");

struct Ctx {
  Bars* bars;
  int* status;
  uint64_t limit_ns;
};

__device__ __forceinline__ void raise(const Ctx& c, int bit) {
  if (c.status) atomicOr(c.status, bit);
}

__device__ __forceinline__ void wait(const Ctx& c, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait(at, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_hint(at, parity, kWaitHintNs)) {
    if (*(volatile int*)&c.bars->abort) return;
    if (globaltimer() - t0 > c.limit_ns) {
      *(volatile int*)&c.bars->abort = 1;
      raise(c, 1);  // MLA_DEVERR_TIMEOUT
      return;
    }
  }
}

__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                       const __grid_constant__ CUtensorMap tm_kv, const KeyWeightArgs a) {
  using S = Shape<kFp8>;
  constexpr int kStages = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + kStages * S::kStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Ctx ctx{bars, a.status, a.wait_limit_ns};
  volatile int* abort_flag = &bars->abort;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars->full[i]), kFp8 ? 5 : 1);   // the loads, and the four expanding warps
      mbar_init(smem_u32(&bars->empty[i]), 1);
      mbar_init(smem_u32(&bars->raw_full[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->d_full[i]), 1);
      mbar_init(smem_u32(&bars->d_empty[i]), 8);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_qr);
    tma_prefetch_desc(&tm_kv);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), 256);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int cap = (int)min((int64_t)a.max_pages * a.page_size, (int64_t)a.weight_len);
  auto keys_of = [&](int b) {
    const int n = a.seq_lens[b];
    return n < 0 ? 0 : (n > cap ? cap : n);
  };
  // this CTA's share of all tiles: a sum over the batch, then the request
  // that holds the share's first tile
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
    long long total = 0, before;
    for (int base = 0; base < a.batch; base += kThreads) {
      const int b = base + tid;
      if (b < a.batch && blockIdx.x == 0 && a.seq_lens[b] > cap) raise(ctx, 2);   // MLA_DEVERR_BAD_SEQ_LEN
      total += block_sum(b < a.batch ? (keys_of(b) + kKeys - 1) / kKeys : 0, before);
    }
    const long long lo = total * blockIdx.x / gridDim.x, hi = total * (blockIdx.x + 1) / gridDim.x;
    long long at = 0;
    for (int base = 0; base < a.batch && at <= lo; base += kThreads) {
      const int b = base + tid;
      const int tiles = b < a.batch ? (keys_of(b) + kKeys - 1) / kKeys : 0;
      const long long all = block_sum(tiles, before);
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
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const int tiles = bars->tiles;
  const int width = a.row_tile;

  auto request = [&](int b) {
    Request r;
    r.n = keys_of(b);
    r.q0 = a.qsl ? a.qsl[b] : b;
    r.sq = a.qsl ? a.qsl[b + 1] - r.q0 : 1;
    if (r.sq < 0 || r.q0 < 0 || r.q0 > a.total_q - r.sq) {
      raise(ctx, 8);   // MLA_DEVERR_BAD_QSL
      r.sq = 0;
    }
    r.rows = r.sq * a.num_heads;
    r.row_tiles = (r.rows + width - 1) / width;
    return r;
  };
  // calls body(request number, request, key tile, whether the request is new) for every tile of the share
  auto for_tiles = [&](auto&& body) {
    int b = bars->b0, t = bars->tile0;
    bool fresh = true;
    Request r{};
    for (int i = 0; i < tiles; ++i, ++t) {
      while (fresh || t * kKeys >= r.n) {
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

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    uint32_t n = 0;
    const int sub_rows = a.page_size < kKeys ? a.page_size : kKeys;
    const int nsub = kKeys / sub_rows;
    const uint64_t pol = l2_policy_evict_first();
    bool skip = a.debug_skip_tile && bars->leads;
    for_tiles([&](int b, const Request& r, int t) {
      // lane l < nsub: the cache row of sub-page l
      int y = (int)(a.num_blocks * a.page_size);   // past the cache: reads zeros
      const int key = t * kKeys + lane * sub_rows;
      if (lane < nsub && key < r.n) {
        const int blk = a.block_table[(int64_t)b * a.max_pages + key / a.page_size];
        if (blk >= 0 && blk < a.num_blocks)
          y = blk * a.page_size + key % a.page_size;
        else
          raise(ctx, 4);   // MLA_DEVERR_BAD_BLOCK
      }
      for (int rt = 0; rt < r.row_tiles; ++rt) {
        const int row0 = r.q0 * a.num_heads + rt * width;
        const int boxes = (min(width, r.rows - rt * width) + a.q_box - 1) / a.q_box;
        for (int c = 0; c < kChunks; ++c, ++n) {
          if (*abort_flag) return;
          const uint32_t slot = n % kStages;
          wait(ctx, &bars->empty[slot], ((n / kStages) & 1) ^ 1);
          __syncwarp();
          if (skip) {      // test aid: the first chunk never comes
            skip = false;
            continue;
          }
          const uint32_t st = smem_u32(smem + slot * S::kStage), full = smem_u32(&bars->full[slot]);
          const uint32_t raw = smem_u32(&bars->raw_full[slot]);
          if (lane == 0) {
            mbar_expect_tx(full, boxes * a.q_box * 128u + (kFp8 ? 0u : kKBytes));
            if (kFp8) mbar_expect_tx(raw, kRawBytes);
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(st + kKBytes + i * a.q_box * 128u, c < 8 ? &tm_q : &tm_qr, c < 8 ? 64 * c : 0,
                          row0 + i * a.q_box, full);
          }
          __syncwarp();
          if (lane < nsub) {
            if (kFp8)
              tma_load_2d_hint(st + kKBytes + kQBytes + lane * sub_rows * 64u, &tm_kv, 64 * c, y, raw, pol);
            else
              tma_load_2d_hint(st + lane * sub_rows * 128u, &tm_kv, 64 * c, y, full, pol);
          }
          __syncwarp();
        }
      }
    });
    // every load has landed before the CTA ends
    for (uint32_t k = n > kStages ? n - kStages : 0; k < n && !*abort_flag; ++k) {
      if (kFp8) wait(ctx, &bars->raw_full[k % kStages], (k / kStages) & 1);
      wait(ctx, &bars->full[k % kStages], (k / kStages) & 1);
    }
  } else if (warp == 1) {
    // --------------------------------------------------------------- products
    const uint32_t hi = desc_hi(1024, kSwizzle128B);
    const uint32_t k_lo = desc_lo(smem_u32(smem), 16), q_lo = desc_lo(smem_u32(smem) + kKBytes, 16);
    uint32_t n = 0, m = 0;
    for_tiles([&](int, const Request& r, int) {
      for (int rt = 0; rt < r.row_tiles; ++rt, ++m) {
        if (*abort_flag) return;
        const uint32_t acc = m & 1;
        const uint32_t cols = (uint32_t)(min(width, r.rows - rt * width) + 15) & ~15u;
        const uint32_t idesc = idesc_bf16_f32(128, cols, 0, 0);
        wait(ctx, &bars->d_empty[acc], ((m >> 1) & 1) ^ 1);
        for (int c = 0; c < kChunks; ++c, ++n) {
          const uint32_t slot = n % kStages;
          wait(ctx, &bars->full[slot], (n / kStages) & 1);
          __syncwarp();
          tc_fence_after();
          if (elect_one()) {
            const uint32_t off = slot * (S::kStage >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ss(tmem + acc * 128, ((uint64_t)hi << 32) | (k_lo + off + 2 * k),
                     ((uint64_t)hi << 32) | (q_lo + off + 2 * k), idesc, (c | k) ? 1u : 0u);
            mma_commit(smem_u32(&bars->empty[slot]));
            if (c == kChunks - 1) mma_commit(smem_u32(&bars->d_full[acc]));
          }
          __syncwarp();
        }
      }
    });
    if (elect_one()) mma_commit(smem_u32(&bars->drain));
    __syncwarp();
    wait(ctx, &bars->drain, 0);
  } else if (warp >= kWarpEpilogue && warp < kWarpExpand) {
    // --------------------------------------------------------------- epilogue
    const int e = tid - 32 * kWarpEpilogue;      // 0..255
    const int q4 = warp & 3, hh = e >> 7;        // tensor-memory lanes 32 q4.., columns of half hh
    const int key = q4 * 32 + lane;
    const uint32_t from = tmem + ((uint32_t)(q4 * 32) << 16);
    uint32_t m = 0, tile_no = 0;
    int at_b = -1;
    uint32_t set = 0;                            // the buffer of lse2 in use
    for_tiles([&](int b, const Request& r, int t) {
      const int j = t * kKeys + key;
      // the first of the request's rows that sees key j (the rest follow)
      const int late = j - (r.n - r.sq);
      const int first_row = late > 0 ? late * a.num_heads : 0;
      const int first_max = __reduce_max_sync(0xffffffffu, first_row);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int rt = 0; rt < r.row_tiles; ++rt, ++m) {
        const uint32_t acc = m & 1;
        const int base = rt * width, cols = min(width, r.rows - base);
        if (r.row_tiles > 1 || at_b != b) {
          set ^= 1;
          if (e < cols) {
            const float l = a.lse[(int64_t)r.q0 * a.num_heads + base + e] * kLog2e;
            bars->lse2[set][e] = l == -INFINITY ? INFINITY : l;   // a row without keys gives no weight
          }
          epilogue_sync();
          at_b = b;
        }
        const float* lse2 = bars->lse2[set];
        wait(ctx, &bars->d_full[acc], (m >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        // 32 columns at a time, the halves in turn
        for (int c0 = 32 * hh; c0 < cols; c0 += 64) {
          uint32_t s[32];
          tmem_ld32(from + acc * 128 + c0, s);
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
        if (lane == 0) mbar_arrive(smem_u32(&bars->d_empty[acc]));
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
  } else if (kFp8 && warp >= kWarpExpand) {
    // -------------------------------------------------------- e4m3 expansion
    const int te = tid - 32 * kWarpExpand;       // 0..127
    uint32_t n = 0;
    for_tiles([&](int, const Request& r, int) {
      for (int i = 0; i < r.row_tiles * kChunks; ++i, ++n) {
        const uint32_t slot = n % kStages;
        wait(ctx, &bars->raw_full[slot], (n / kStages) & 1);
        __syncwarp();
        const uint8_t* st = smem + slot * S::kStage;
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = reinterpret_cast<const uint4*>(st + kKBytes + kQBytes)[te + 128 * k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = te + 128 * k, q = at & 3, row = at >> 2;
          uint32_t o[8];
          widen16(v[k], o);
          uint4* dst = reinterpret_cast<uint4*>(smem + slot * S::kStage + row * 128);
          dst[(2 * q) ^ (row & 7)] = make_uint4(o[0], o[1], o[2], o[3]);
          dst[(2 * q + 1) ^ (row & 7)] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->full[slot]));
      }
    });
  }
  __syncwarp();
  if (*abort_flag) {
    // given up: loads and products in flight finish well within this time
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <bool kFp8>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_qr, const CUtensorMap& tm_kv, const KeyWeightArgs& a,
                   int sm_count, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(key_weights_kernel<kFp8>, Shape<kFp8>::kSmem, done);
  if (e != cudaSuccess) return e;
  // no more CTAs than tiles there can be
  const int64_t reach = (int64_t)a.max_pages * a.page_size < a.weight_len ? (int64_t)a.max_pages * a.page_size
                                                                          : (int64_t)a.weight_len;
  const int64_t most = a.batch * ((reach + kKeys - 1) / kKeys);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < sm_count ? (most > 0 ? most : 1) : sm_count));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<kFp8>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, key_weights_kernel<kFp8>, tm_q, tm_qr, tm_kv, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_key_weights(const CUtensorMap& tm_q, const CUtensorMap& tm_qr, const CUtensorMap& tm_kv, int fp8,
                               const KeyWeightArgs& a, int sm_count, cudaStream_t s) {
  return fp8 ? launch<true>(tm_q, tm_qr, tm_kv, a, sm_count, s) : launch<false>(tm_q, tm_qr, tm_kv, a, sm_count, s);
}

}  // namespace mla
