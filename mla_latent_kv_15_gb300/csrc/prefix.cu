// Attention of many query rows over a shared prefix (mla_decode_shared), on
// tcgen05:  partial out and lse of the rows of all requests behind a prefix
// over a range of its keys,  s = scale q.k,  out = sum softmax(s) kv_c.
//
// The decode kernel holds 128 rows' 512-wide output in the tensor memory of two
// CTAs, each with half of its columns, and exchanges partial scores.  That is
// right where a request's 128 rows read their keys from HBM; a prefix is read
// from L2 by one group of 128 rows after the other, and the products count.
// Here both products have the long side of the tile as their rows:
//
//   S = K . Q^T    256 keys x 128 query rows, 576 deep
//   O = V^T . P    512 latent dims x 128 query rows, 256 keys deep
//
// as pair products (cta_group::2): a CTA has 128 of the tile's keys as rows of S
// and 2 x 128 of the latent dims as rows of O, and half of the query rows as
// columns of either operand.  O is 256 columns of tensor memory, S two buffers
// of 128.  A thread of the softmax has one key and 64 query rows; it writes its
// probabilities as rows of P^T, 64 rows wide in the CTA that multiplies them, and
// adds them up in registers, reduced over keys when the unit ends.
//
// No running maximum: exponents are relative to a reference, the largest score
// of the row among the first 32 keys of the unit's range, and bf16 and float32
// carry 2^+-126 either way.  Keys further below underflow beside the one that
// gave the reference.  A row whose sum passes 2^80 (a later score is 55 above the
// reference, in natural units) marks its unit, which the decode kernel, launched
// next for the requests' own keys, does again with its running maximum.
//
// Operands stream through a ring of 16 KB slots: nine 64-column chunks of the
// CTA's keys for S, then eight 64-key x 128-dim boxes of all 256 keys for O; the
// next tile's S runs before a tile's O, so that the softmax has its time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                     // keys of a CTA's half of a tile
constexpr int kChunks = kDqk / 64;             // 9
constexpr int kValueItems = 2 * kPrefixTile / 64;   // two 128-dim halves x four groups of 64 keys
constexpr uint32_t kSlot = 16384;
constexpr int kSlots = 7;
constexpr uint32_t kQChunk = 64 * 128;         // 64 query rows x 64 columns
constexpr uint32_t kQBytes = kChunks * kQChunk;
constexpr uint32_t kPBytes = kPrefixTile * 128;   // 256 keys x 64 rows bf16
constexpr int kThreads = 384;                  // warp 0 loads, 1 issues, 2 owns tensor memory, 4-11 softmax
constexpr int kWarpLoad = 0, kWarpMma = 1, kWarpTmem = 2, kWarpSoftmax = 4;
constexpr uint32_t kColO = 0, kColS = 256;     // O halves, S buffers: 128 columns each
constexpr float kMaxSum = 1.2089258e24f;       // 2^80

// Barriers marked (lead) are used in the leading CTA only, by both CTAs.
struct Bars {
  uint64_t full[kSlots];      // (lead) both CTAs' halves are there
  uint64_t empty[kSlots];
  uint64_t tail;              // values with rows behind the last key have landed
  uint64_t q_full;            // (lead)
  uint64_t q_free;            // the unit's last S is computed
  uint64_t s_full[2];
  uint64_t p_full;            // (lead) the softmax warps of both CTAs
  uint64_t p_free;            // a tile's O is added
  uint64_t o_full;
  uint64_t o_free;            // (lead) the softmax warps of both CTAs have read O
  uint64_t ref_full;          // the unit's references are here
  uint64_t sum_full;          // every warp's sums are here
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  // (a warp writes those of the next unit only when all have used the last's)
  alignas(16) float ref[128];      // a row's reference, scaled
  float sums[8][128];              // [CTA, lane quadrant][row]
  float inv[8][64];                // of a warp's 64 rows
};
constexpr size_t kSmem = 1024 + kQBytes + kPBytes + kSlots * kSlot + sizeof(Bars);
static_assert(kSmem <= 232448, "shared memory per CTA");

struct Ctx {
  Bars* bars;
  int* status;
  uint64_t limit_ns;
};

__device__ __forceinline__ void give_up(const Ctx& c) {
  *(volatile int*)&c.bars->abort = 1;
  atomicOr(c.status, 1);   // MLA_DEVERR_TIMEOUT
}
// Bounded waits; once the CTA has given up they return at once.
__device__ __forceinline__ void wait(const Ctx& c, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait(at, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_hint(at, parity, kWaitHintNs)) {
    if (*(volatile int*)&c.bars->abort) return;
    if (globaltimer() - t0 > c.limit_ns) return give_up(c);
  }
}
// The same for what the other CTA has written.
__device__ __forceinline__ void wait_cluster(const Ctx& c, uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait_cluster(at, parity)) return;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_cluster_hint(at, parity, kWaitHintNs)) {
    if (*(volatile int*)&c.bars->abort) return;
    if (globaltimer() - t0 > c.limit_ns) return give_up(c);
  }
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n"
      " mov.b64 {%0, %1}, x;\n}" : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}
// a float's order-preserving unsigned code, and back
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t u = __float_as_uint(x);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t c) {
  return __uint_as_float(c & 0x80000000u ? c ^ 0x80000000u : ~c);
}

__device__ __forceinline__ void st_cluster_v4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qr,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_smem = smem;
  uint8_t* p_smem = smem + kQBytes;
  uint8_t* ring = p_smem + kPBytes;
  Bars* bars = reinterpret_cast<Bars*>(ring + kSlots * kSlot);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = (int)cluster_id_x();
  const Plan& P = a.prefix;
  const Ctx ctx{bars, &P.header->status, a.wait_limit_ns};
  volatile int* abort_flag = &bars->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&bars->full[i]), 2);
      mbar_init(smem_u32(&bars->empty[i]), 1);
    }
    mbar_init(smem_u32(&bars->tail), 1);
    mbar_init(smem_u32(&bars->q_full), 2);
    mbar_init(smem_u32(&bars->q_free), 1);
    mbar_init(smem_u32(&bars->s_full[0]), 1);
    mbar_init(smem_u32(&bars->s_full[1]), 1);
    mbar_init(smem_u32(&bars->p_full), 16);
    mbar_init(smem_u32(&bars->p_free), 1);
    mbar_init(smem_u32(&bars->o_full), 1);
    mbar_init(smem_u32(&bars->o_free), 16);
    mbar_init(smem_u32(&bars->ref_full), 2);
    mbar_init(smem_u32(&bars->sum_full), 16);
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_qr);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kWarpTmem) {
    tmem_alloc_pair(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are initialised before either uses the other's
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ubeg = P.cluster_begin[pair], uend = P.cluster_begin[pair + 1];

  if (warp == kWarpLoad) {
    // ------------------------------------------------------------------ loads
    uint32_t n = 0, tails = 0, units = 0;
    const int krows = a.page_size < kKeys ? a.page_size : kKeys, vrows = a.page_size < 64 ? a.page_size : 64;
    const int past = a.num_blocks * a.page_size;     // reads zeros
    const uint64_t pol = l2_policy_evict_last();     // the next group of rows reads the prefix again
    bool skip = a.debug_skip_tile && pair == 0 && rank == 0;
    auto next_slot = [&]() {
      const uint32_t slot = n % kSlots;
      wait(ctx, &bars->empty[slot], ((n / kSlots) & 1) ^ 1);
      ++n;
      __syncwarp();
      return slot;
    };
    for (int u = ubeg; u < uend; ++u, ++units) {
      const UnitRec ur = P.units[u];
      const int32_t* table = a.prefix_table + (int64_t)~ur.b * a.max_prefix_pages;
      auto row_of = [&](int key) {
        if (key >= ur.lmax) return past;
        const int blk = table[key / a.page_size];
        if (blk >= 0 && blk < a.num_blocks) return blk * a.page_size + key % a.page_size;
        atomicOr(ctx.status, 4);   // MLA_DEVERR_BAD_BLOCK
        return past;
      };
      // the CTA's 64 query rows, once the last unit's scores are computed
      wait(ctx, &bars->q_free, (units & 1) ^ 1);
      __syncwarp();
      if (elect_one()) {
        const uint32_t full = mapa(smem_u32(&bars->q_full), 0);
        mbar_expect_tx_remote(full, kQBytes);
        for (int c = 0; c < kChunks; ++c)
          tma_load_2d_pair(smem_u32(q_smem + c * kQChunk), c < 8 ? &tm_q : &tm_qr, c < 8 ? 64 * c : 0,
                           ur.row0 + 64 * (int)rank, full);
      }
      __syncwarp();
      // the nine chunks of the CTA's keys of tile t
      auto load_keys = [&](int t) {
        const int y = lane * krows < kKeys ? row_of(t * kPrefixTile + kKeys * (int)rank + lane * krows) : past;
        for (int c = 0; c < kChunks; ++c) {
          if (*abort_flag) return;
          const uint32_t slot = next_slot();
          if (skip) {              // test aid: the first chunk never comes
            skip = false;
            continue;
          }
          const uint32_t full = mapa(smem_u32(&bars->full[slot]), 0);
          if (lane == 0) mbar_expect_tx_remote(full, kSlot);
          __syncwarp();
          if (lane * krows < kKeys)
            tma_load_2d_pair_hint(smem_u32(ring + slot * kSlot) + lane * krows * 128u, &tm_k, 64 * c, y, full, pol);
          __syncwarp();
        }
      };
      // the eight boxes of the tile's values: the CTA's 128 dims of either half
      // of the latent row, four groups of 64 keys
      auto load_values = [&](int t) {
        const int y = lane * vrows < kPrefixTile ? row_of(t * kPrefixTile + lane * vrows) : past;
        for (int i = 0; i < kValueItems; ++i) {
          if (*abort_flag) return;
          const int x = 256 * (i >> 2) + 128 * (int)rank, key0 = t * kPrefixTile + 64 * (i & 3);
          const int box = lane - (i & 3) * (64 / vrows);     // the lane's box of the group
          const bool mine = box >= 0 && box < 64 / vrows;
          const uint32_t slot = next_slot();
          const uint32_t full = mapa(smem_u32(&bars->full[slot]), 0), dst = smem_u32(ring + slot * kSlot);
          const int live = ur.lmax - key0;
          if (live > 0 && live < 64) {
            // rows behind the last key: their probabilities are zero, but what
            // the page holds there may be infinite or NaN
            const uint32_t tail = smem_u32(&bars->tail);
            if (lane == 0) mbar_expect_tx(tail, kSlot);
            __syncwarp();
            if (mine)
              for (int d = 0; d < 2; ++d) tma_load_2d(dst + d * 8192 + box * vrows * 128u, &tm_v, x + 64 * d, y, tail);
            wait(ctx, &bars->tail, tails++ & 1);
            __syncwarp();
            for (int d = 0; d < 2; ++d)
              for (int at = live * 128 + lane * 16; at < 64 * 128; at += 32 * 16)
                *reinterpret_cast<uint4*>(ring + slot * kSlot + d * 8192 + at) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_release_cluster(full);
          } else {
            if (lane == 0) mbar_expect_tx_remote(full, kSlot);
            __syncwarp();
            if (mine)
              for (int d = 0; d < 2; ++d)
                tma_load_2d_pair_hint(dst + d * 8192 + box * vrows * 128u, &tm_v, x + 64 * d, y, full, pol);
          }
          __syncwarp();
        }
      };
      load_keys(ur.tile_begin);
      for (int t = ur.tile_begin; t < ur.tile_end; ++t) {
        if (t + 1 < ur.tile_end) load_keys(t + 1);
        load_values(t);
      }
    }
    // every load of the pair has landed before it ends
    if (rank == 0)
      for (uint32_t k = n > kSlots ? n - kSlots : 0; k < n && !*abort_flag; ++k)
        wait(ctx, &bars->full[k % kSlots], (k / kSlots) & 1);
  } else if (warp == kWarpMma) {
    // --------------------------------------------------------------- products
    if (rank == 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(256, 128, 0, 0), id_o = idesc_bf16_f32(256, 128, 1, 1);
      constexpr uint32_t hi = desc_hi(1024, kSwizzle128B);
      const uint32_t ring_k = desc_lo(smem_u32(ring), 16), ring_v = desc_lo(smem_u32(ring), 8192);
      const uint32_t q_lo = desc_lo(smem_u32(q_smem), 16), p_lo = desc_lo(smem_u32(p_smem), 8192);
      uint32_t n = 0, tile = 0, units = 0, s_tile = 0;
      for (int u = ubeg; u < uend; ++u, ++units) {
        const UnitRec ur = P.units[u];
        wait(ctx, &bars->q_full, units & 1);
        // S's buffer is free: its tile before last has its probabilities written
        auto scores = [&](bool last) {
          const uint32_t d = tmem + kColS + (s_tile & 1) * 128;
          for (int c = 0; c < kChunks; ++c, ++n) {
            const uint32_t slot = n % kSlots;
            wait(ctx, &bars->full[slot], (n / kSlots) & 1);
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t ka = ring_k + slot * (kSlot >> 4), qa = q_lo + c * (kQChunk >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_pair_ss(d, ka + 2 * k, hi, qa + 2 * k, hi, id_s, (c | k) ? 1u : 0u);
              mma_commit_pair(smem_u32(&bars->empty[slot]));
              if (c == kChunks - 1) {
                mma_commit_pair(smem_u32(&bars->s_full[s_tile & 1]));
                if (last) mma_commit_pair(smem_u32(&bars->q_free));
              }
            }
            __syncwarp();
          }
          ++s_tile;
        };
        const int nt = ur.tile_end - ur.tile_begin;
        scores(nt == 1);
        for (int t = 0; t < nt; ++t, ++tile) {
          if (*abort_flag) break;
          if (t + 1 < nt) scores(t + 2 == nt);
          wait_cluster(ctx, &bars->p_full, tile & 1);
          if (t == 0) wait(ctx, &bars->o_free, (units & 1) ^ 1);
          fence_proxy_async();
          for (int i = 0; i < kValueItems; ++i, ++n) {
            const uint32_t slot = n % kSlots;
            wait_cluster(ctx, &bars->full[slot], (n / kSlots) & 1);
            __syncwarp();
            tc_fence_after();
            if (elect_one()) {
              const uint32_t va = ring_v + slot * (kSlot >> 4), pa = p_lo + (i & 3) * (64 * 128 >> 4);
              const uint32_t d = tmem + kColO + (i >> 2) * 128;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_pair_ss(d, va + 128 * k, hi, pa + 128 * k, hi, id_o, t > 0 || (i & 3) || k ? 1u : 0u);
              mma_commit_pair(smem_u32(&bars->empty[slot]));
              if (i == kValueItems - 1) {
                mma_commit_pair(smem_u32(&bars->p_free));
                if (t == nt - 1) mma_commit_pair(smem_u32(&bars->o_full));
              }
            }
            __syncwarp();
          }
        }
      }
      if (elect_one()) mma_commit_pair(smem_u32(&bars->drain));
      __syncwarp();
      wait(ctx, &bars->drain, 0);
    }
  } else if (warp >= kWarpSoftmax) {
    // ---------------------------------------------------------------- softmax
    const int w = warp - kWarpSoftmax;
    const int q4 = warp & 3, hh = w >> 2;          // tensor-memory lanes 32 q4.., rows 64 hh..
    const int key = q4 * 32 + lane;                // of the CTA's 128
    const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
    const uint32_t from_s = tmem + kColS + 64 * hh + lanes;
    const int tile_key = kKeys * (int)rank + key;  // of the tile's 256
    // this key's row of P^T, in the CTA that has rows 64 hh.. as its columns
    const uint32_t p_row = mapa(smem_u32(p_smem), (uint32_t)hh) + tile_key * 128;
    uint32_t tile = 0, units = 0;
    for (int u = ubeg; u < uend; ++u, ++units) {
      const UnitRec ur = P.units[u];
      const uint32_t set = units & 1;
      const int kend = min(ur.tile_end * kPrefixTile, ur.lmax);
      const float* ref = bars->ref + 64 * hh;
      float sum[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) sum[c] = 0.f;
      for (int t = ur.tile_begin; t < ur.tile_end; ++t, ++tile) {
        wait(ctx, &bars->s_full[tile & 1], (tile >> 1) & 1);
        __syncwarp();
        tc_fence_after();
        const uint32_t s_at = from_s + (tile & 1) * 128;
        const bool live = t * kPrefixTile + tile_key < kend;
        if (t == ur.tile_begin) {
          if (rank == 0 && q4 == 0) {
            // the references: the largest score among the unit's first 32 keys
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              uint32_t s[32];
              tmem_ld32(s_at + 32 * g, s);
              tmem_wait_ld();
              float mine = 0.f;
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, live ? order(__uint_as_float(s[c]) * a.scale_log2) : 0u);
                if (lane == c) mine = unorder(top);
              }
              const int row = 64 * hh + 32 * g + lane;
              for (uint32_t r = 0; r < 2; ++r) st_cluster(mapa(smem_u32(&bars->ref[row]), r), mine);
            }
            __syncwarp();
            if (lane < 2) mbar_arrive_release_cluster(mapa(smem_u32(&bars->ref_full), lane));
          }
          wait_cluster(ctx, &bars->ref_full, set);
          __syncwarp();
        }
        uint32_t pk[32];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t s[32];
          tmem_ld32(s_at + 32 * g, s);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 m = *reinterpret_cast<const float4*>(ref + 32 * g + c);
            float p0 = exp2_fast(fmaf(__uint_as_float(s[c]), a.scale_log2, -m.x));
            float p1 = exp2_fast(fmaf(__uint_as_float(s[c + 1]), a.scale_log2, -m.y));
            float p2 = exp2_fast(fmaf(__uint_as_float(s[c + 2]), a.scale_log2, -m.z));
            float p3 = exp2_fast(fmaf(__uint_as_float(s[c + 3]), a.scale_log2, -m.w));
            p0 = live ? p0 : 0.f;
            p1 = live ? p1 : 0.f;
            p2 = live ? p2 : 0.f;
            p3 = live ? p3 : 0.f;
            add2(sum[32 * g + c], sum[32 * g + c + 1], p0, p1);
            add2(sum[32 * g + c + 2], sum[32 * g + c + 3], p2, p3);
            pk[16 * g + c / 2] = pack_bf16x2(p0, p1);
            pk[16 * g + c / 2 + 1] = pack_bf16x2(p2, p3);
          }
        }
        // (a score buffer is free again once its probabilities are announced)
        tc_fence_before();
        wait(ctx, &bars->p_free, (tile & 1) ^ 1);   // the tile before has been multiplied
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_cluster_v4(p_row + ((uint32_t)(i ^ (tile_key & 7)) << 4), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2],
                        pk[4 * i + 3]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive_release_cluster(mapa(smem_u32(&bars->p_full), 0));
      }
      // sums over the warp's keys: lane l gets rows 2 l and 2 l + 1 (halves of
      // the rows go to the partner, five times)
#pragma unroll
      for (int o = 16, half = 32; o >= 1; o >>= 1, half >>= 1) {
        const bool upper = lane & o;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (c < half) {
            const float keep = upper ? sum[half + c] : sum[c], give = upper ? sum[c] : sum[half + c];
            sum[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
      }
      const int row2 = 64 * hh + 2 * lane;
      for (uint32_t r = 0; r < 2; ++r) {
        const uint32_t to = mapa(smem_u32(&bars->sums[4 * rank + q4][row2]), r);
        st_cluster(to, sum[0]);
        st_cluster(to + 4, sum[1]);
      }
      __syncwarp();
      if (lane < 2) mbar_arrive_release_cluster(mapa(smem_u32(&bars->sum_full), lane));
      wait_cluster(ctx, &bars->sum_full, set);
      __syncwarp();
      float* inv = bars->inv[w];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float l = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) l += bars->sums[i][row2 + k];
        inv[2 * lane + k] = 1.f / l;
        if (row2 + k < ur.nrows) {
          if (!(l < kMaxSum)) P.redo[u] = 1;       // (NaN too)
          if (rank == 0 && q4 == 0)
            P.part_lse[(size_t)ur.slot * kRows + row2 + k] = (bars->ref[row2 + k] + __log2f(l)) * 0.6931471805599453f;
        }
      }
      __syncwarp();
      wait(ctx, &bars->o_full, set);
      __syncwarp();
      tc_fence_after();
      // O: the thread has dims 256 h + 128 rank + 32 q4 + lane of the warp's 64
      // rows.  fp16 codes with one power of two for the 32 dims of a warp and
      // row, as the decode kernel's partials; lanes in pairs store two dims of
      // one row each.
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        const int h = g >> 1, c0 = 32 * (g & 1);
        uint32_t o[32];
        tmem_ld32(tmem + kColO + 128 * h + 64 * hh + c0 + lanes, o);
        tmem_wait_ld();
        const int chunk = 8 * h + 4 * (int)rank + q4;
        float scale = 0.f;
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          uint32_t code[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float v = __uint_as_float(o[c + k]) * inv[c0 + c + k];
            const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v)));
            const int mexp = min(253, 268 - (int)(top >> 23));
            code[k] = __half_as_ushort(__float2half_rn(v * __int_as_float(mexp << 23)));
            if (lane == c + k) scale = __int_as_float((254 - mexp) << 23);
          }
          const bool odd = lane & 1;
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? code[0] : code[1], 1);
          const uint32_t word = odd ? got | code[1] << 16 : code[0] | got << 16;
          const int row = 64 * hh + c0 + c + odd;
          if (row < ur.nrows)
            *reinterpret_cast<uint32_t*>(P.part_o + ((size_t)ur.slot * kRows + row) * kLkv + 32 * chunk + (lane & ~1)) = word;
        }
        const int row = 64 * hh + c0 + lane;
        if (row < ur.nrows) P.part_scale[((size_t)ur.slot * kRows + row) * (kLkv / 32) + chunk] = scale;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&bars->o_free), 0));
    }
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
  cluster_sync();   // the pair ends together: each reads, writes and signals the other's shared memory
  if (warp == kWarpTmem) {
    // the last signal to the peer's own barriers is on its way by now
    if (rank == 1) wait(ctx, &bars->drain, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_prefix(const CUtensorMap& tm_q, const CUtensorMap& tm_qr, const CUtensorMap& tm_k,
                          const CUtensorMap& tm_v, const DecodeArgs& a, int num_clusters, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(prefix_kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)num_clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefix_kernel, tm_q, tm_qr, tm_k, tm_v, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
