// Expanded latent attention (mla_prefill) on tcgen05: packed sequences, every
// head with its own 128-wide key and value and one 64-wide rotated key shared
// by all heads.
//
//   s_ij = scale * (q_nope_i . k_nope_j + q_pe_i . k_pe_j)
//   out_i = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i)
//
// A pair of CTAs takes items (512 query rows of a head x a range of keys): a
// product of the pair has 256 query rows, 128 in each CTA, against keys and
// values of which each CTA holds half (64 of a tile's 128 keys for the scores,
// 64 of the 128 value dims for the outputs), so that a key is loaded once for
// 512 queries and shared memory has room for three tiles beside the queries
// (a single-CTA form, with room for 1.6, waited for loads a third of the
// time: 8192-token prompt of 128 heads, 2245 us).  Tensor memory of each CTA:
// scores S0, S1 and outputs O0, O1, 128 columns each; a tile's
// probabilities (bf16) overwrite its scores.  One thread of the leading CTA
// issues, per key tile,
//   O0 += P0 V_j,  S0 = Q0 K_{j+1},  O1 += P1 V_j,  S1 = Q1 K_{j+1}
// so the tensor cores work on one query tile while the softmax warps of the
// other turn its scores into probabilities.  The softmax thread of a row
// keeps the running reference m and sum in float32 and scales O in place,
// but only when a row's maximum has risen by more than 2^8 over the
// reference, which leaves the result the same and is rare.  P is rounded to
// bf16 for the product (the sum is of the unrounded values).
//
// An item of up to 256 rows ("narrow") has one query tile: the pair takes its
// even key tiles as tile 0 and its odd ones as tile 1, so that the two still
// work in turn, and the warps of tile 0 join the two results at the end.
//
// Measured (128 heads): causal prompt of 8192 tokens 1650 us back to back, 1666
// TFLOP/s, 98 % of the library's matrix rate under the same power cap; 512 rows
// over 16384 keys without a mask 428 us, 1605 TFLOP/s; eight single tokens over
// up to 8191 keys of 16 heads 55 us, 4.1 TB/s.  A step of a query tile takes
// ~1430 cycles, its products at least 1280; short prompts lose ~4000 cycles an
// item and ~2000 on each key tile that tile 1 has alone (16 prompts of 1024, 32
// heads: 182 us, half of it products).  Two threads a row (16 softmax warps of
// 96 registers) were slower: 8192 tokens 1840 us, 16 prompts of 1024 199.
#include <cuda_bf16.h>

#include "common.cuh"
#include "prefill.cuh"
#include "ptx.cuh"

namespace mla {
namespace {
using namespace ptx;

constexpr int kSoftmaxWarps = 8;                  // 0-3: query tile 0, 4-7: query tile 1
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarpList = 10, kWarpClear = 11;
constexpr int kItemSlots = 2;                     // items known ahead
constexpr int kItemReaders = 2 * (kSoftmaxWarps + 2) + 2;   // both CTAs' softmax, load and clearing warps, the MMA warp, the peer's list warp
constexpr int kThreads = 384;
constexpr uint32_t kRegsSoftmax = 216, kRegsOther = 72;
static_assert(128 * (2 * kRegsSoftmax + kRegsOther) <= kThreads * 168, "register split of the launch's 168 a thread");

constexpr uint32_t kQChunk = 16384;               // 128 rows x 64 dims
constexpr uint32_t kQTile = 3 * kQChunk;
constexpr uint32_t kBox = 8192;                   // 64 rows x 64 dims: one load of keys or values
constexpr uint32_t kKeyBytes = 3 * kBox;          // the CTA's 64 keys of a tile
constexpr uint32_t kValueBytes = 2 * kBox;        // the CTA's 64 value dims of a tile's 128 keys
constexpr uint32_t kStage = kKeyBytes + kValueBytes;
constexpr int kStages = 3;
constexpr uint32_t kColS = 0, kColO = 256;        // S0 S1 O0 O1
constexpr float kRescale = 8.0f;                  // log2 units

// Barriers marked (lead) are used in the leading CTA only, by both CTAs.
struct Bars {
  uint64_t k_full[kStages], v_full[kStages];      // (lead) both CTAs' halves have landed
  uint64_t k_empty[kStages], v_empty[kStages];
  uint64_t v_tail[kStages];                       // the CTA's half of a value tile with rows to clear has landed
  uint64_t q_full[2];                             // (lead)
  uint64_t q_empty[2];
  uint64_t s_full[2], o_full[2];
  uint64_t p_full[2];                             // (lead) all softmax warps of the pair
  uint64_t x_full[4], x_done[4];                  // narrow items: rows of a quadrant of tile 1 handed over, and read
  uint64_t drain;
  uint64_t item_full[kItemSlots];
  uint64_t item_empty[kItemSlots];                // (lead)
  uint32_t tmem_base;
  int abort;
  int mending;                                    // warps of the pair that compute rows again (mend_row)
};
constexpr size_t kSmem = 1024 + 2 * kQTile + kStages * kStage + sizeof(Bars) + 16 + kItemSlots * 48 + 128 * 8;
static_assert(kSmem <= 232448, "shared memory per CTA");

struct Ctx {
  Bars* bars;
  uint32_t rank;      // in the pair; 0 leads
  uint64_t limit_ns;
  // shared::cluster address of the leading CTA's copy of one of `bars`
  __device__ __forceinline__ uint32_t lead(uint64_t* bar) const { return mapa(smem_u32(bar), 0); }
};

// Bounded waits; once one has run out, every other one of the CTA returns, and
// the peer's run out in turn; the CTA reports it when it ends.  The time in which rows are mended, which ends by
// itself but may be long, does not count.  kCluster: the acquire covers what the other CTA
// has written to shared memory.  Waits for an item, or for its last keys, may
// last as long as an item (`times` the limit).
template <bool kCluster = false>
__device__ __forceinline__ void wait_bar(const Ctx& c, uint64_t* bar, uint32_t parity, uint32_t times = 1) {
  const uint32_t at = smem_u32(bar);
  if (kCluster ? mbar_try_wait_cluster(at, parity) : mbar_try_wait(at, parity)) return;
  uint64_t t0 = globaltimer();
  while (!(kCluster ? mbar_try_wait_cluster_hint(at, parity, kWaitHintNs) : mbar_try_wait_hint(at, parity, kWaitHintNs))) {
    if (*(volatile int*)&c.bars->abort) return;
    if (*(volatile int*)&c.bars->mending) t0 = globaltimer();
    if (globaltimer() - t0 > c.limit_ns * times) {
      *(volatile int*)&c.bars->abort = 1;
      return;
    }
  }
}
constexpr uint32_t kItemWait = 64;

// The pair's count of warps that mend rows, kept in both CTAs.
__device__ __noinline__ void count_mending(const Ctx& c, int lane, int step) {
  __syncwarp();
  if (lane < 2)
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(mapa(smem_u32(&c.bars->mending), lane)),
                 "r"(step)
                 : "memory");
  __syncwarp();
}

struct __align__(16) Item {
  int q0, nq, kv0, nkeys, lim0, prow, head;
  int seen[2];     // keys the last row of each query tile sees (0: no such row)
  int tiles[2];    // their key tiles
  int last;        // behind the last item: nothing to do
};
static_assert(sizeof(Item) == 48, "three 16-byte words");

// Whether the item has one query tile, whose key tiles alternate between the
// two: key tile of step i of tile t.
__device__ __forceinline__ bool narrow_item(const Item& it) { return it.nq <= kPrefillRows / 2; }
__device__ __forceinline__ int key_tile(bool narrow, int t, int i) { return narrow ? 2 * i + t : i; }
// Key tiles in all.
__device__ __forceinline__ int tiles_of(const Item& it) {
  return narrow_item(it) ? it.tiles[0] + it.tiles[1] : max(it.tiles[0], it.tiles[1]);
}

// What follows from an item's rows and keys.
__device__ __forceinline__ void finish_item(const PrefillArgs& a, Item& it) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(256 * (t + 1), it.nq) - 1;
    it.seen[t] = it.nq > 256 * t ? min(max(it.lim0 + (a.causal ? last : 0), 0), it.nkeys) : 0;
    it.tiles[t] = (it.seen[t] + kPrefillTile - 1) / kPrefillTile;
  }
  if (narrow_item(it)) {
    it.seen[1] = it.seen[0];
    it.tiles[1] = it.tiles[0] / 2;
    it.tiles[0] -= it.tiles[1];
  }
  it.last = 0;
}

// Item `i` of the list: pieces longest first, interleaved over a group of
// heads; in a fixed plan a piece is an item.
__device__ __forceinline__ Item item_at(const PrefillArgs& a, int np, int group, bool fixed, int i) {
  int p = i, head = 0;
  if (!fixed) {
    const int per = np * group;               // <= items, which are below 2^31
    const int g = i / per, rem = i - g * per;
    const int heads = min(group, a.num_heads - g * group);
    p = rem / heads;
    head = g * group + rem - p * heads;
  }
  const int4* rec = reinterpret_cast<const int4*>(a.plan.pieces + p);
  const int4 r0 = rec[0], r1 = rec[1];
  Item it;
  it.q0 = r0.x, it.nq = r0.y, it.kv0 = r0.z, it.nkeys = r0.w, it.lim0 = r1.x, it.prow = r1.y;
  it.head = fixed ? r1.z : head;
  if (it.prow >= 0) it.prow += head * it.nq;
  finish_item(a, it);
  return it;
}

// Item `i` without a plan, by the whole warp: lane b holds sequence b (`seq`:
// its first rows and lengths) and the blocks before it.
__device__ __forceinline__ Item item_direct(const PrefillArgs& a, const int4 seq, int before, int blocks, int i) {
  const int blk = i / a.num_heads;
  const unsigned owner = __ballot_sync(0xffffffffu, blk >= before && blk < before + blocks);
  const int src = __ffs(owner) - 1;
  const int r0 = (blk - __shfl_sync(0xffffffffu, before, src)) * kPrefillRows;
  const PrefillBlock b = prefill_block(__shfl_sync(0xffffffffu, seq.x, src), __shfl_sync(0xffffffffu, seq.y, src),
                                       __shfl_sync(0xffffffffu, seq.z, src), __shfl_sync(0xffffffffu, seq.w, src), r0,
                                       a.causal);
  Item it;
  it.q0 = b.q0, it.nq = b.nq, it.kv0 = b.kv0, it.nkeys = b.nkeys, it.lim0 = b.lim0, it.prow = -1;
  it.head = i - blk * a.num_heads;
  finish_item(a, it);
  return it;
}

// A pair's span of all items laid end to end (head after head, `all` units
// each; lane b: sequence b's units and those before it).
struct Span {
  int from, to;           // [from, to)
  int at;                 // where item (head, sequence src, row r0) begins
  int head, src, r0;
};

__device__ __forceinline__ PrefillBlock span_block(const PrefillArgs& a, const int4 seq, const Span& p) {
  return prefill_block(__shfl_sync(0xffffffffu, seq.x, p.src), __shfl_sync(0xffffffffu, seq.y, p.src),
                       __shfl_sync(0xffffffffu, seq.z, p.src), __shfl_sync(0xffffffffu, seq.w, p.src), p.r0, a.causal);
}
// Behind the item of `cost` units at p.at.
__device__ __forceinline__ void span_advance(Span& p, int cost, int rows, unsigned filled) {
  p.at += kPrefillItemUnits + cost;
  p.r0 += kPrefillRows;
  if (p.r0 < rows) return;
  p.r0 = 0;
  const unsigned later = p.src == 31 ? 0 : filled & ~((2u << p.src) - 1);
  p.head += later == 0;
  p.src = __ffs(later ? later : filled) - 1;
}
// The span's next piece, by the whole warp; behind its end, it.last.  The
// first piece of an item that ends in another span is noted for the join.
__device__ __forceinline__ void span_next(const PrefillArgs& a, const int4 seq, Span& p, unsigned filled, int length,
                                       int used, int pair, Item& it) {
  it.last = 1;
  while (p.at < p.to && it.last) {
    const PrefillBlock b = span_block(a, seq, p);
    const int tiles = b.tiles(), unit = b.unit(), rows = __shfl_sync(0xffffffffu, seq.y, p.src);
    const int end = p.at + kPrefillItemUnits + b.cost();
    const int t0 = prefill_tiles_before(p.from, p.at, unit, tiles);
    const int t1 = end <= p.to ? tiles : prefill_tiles_before(p.to, p.at, unit, tiles);
    if (t1 > t0 || (end <= p.to && tiles == 0)) {
      it.q0 = b.q0, it.nq = b.nq, it.kv0 = b.kv0 + t0 * kPrefillTile, it.lim0 = b.lim0 - t0 * kPrefillTile;
      it.nkeys = min(t1 * kPrefillTile, b.nkeys) - t0 * kPrefillTile;
      it.head = p.head;
      const int own = 2 * pair + (t0 == 0), first = prefill_span_rows(a.total_q) * own;
      it.prow = t0 == 0 && t1 == tiles ? -1 : first;
      if (t0 == 0 && t1 < tiles && (threadIdx.x & 31) == 0) {
        PrefillSplit sp{};
        sp.q0 = b.q0, sp.nq = b.nq, sp.head0 = p.head, sp.heads = 1, sp.prow = first;
        sp.stride = 2 * prefill_span_rows(a.total_q);
        // up to the first span that ends at `end` or behind it; no span between is without a tile
        // (a span is at least as long as an empty item, 3 units, a tile 2)
        sp.pieces = (int)(((unsigned)end * used + length - 1) / (unsigned)length) - pair;
        a.plan.splits[pair] = sp;
      }
      finish_item(a, it);
    }
    span_advance(p, b.cost(), rows, filled);
  }
}

// The leading CTA's list warp hands the pair's item number n to both CTAs.
// Returns whether it was the last (a last one tells the peer of an abort, too).
__device__ __forceinline__ bool hand_item(const Ctx& ctx, Item* slots, int lane, uint32_t n, Item& it) {
  Bars* bars = ctx.bars;
  const uint32_t slot = n % kItemSlots;
  wait_bar(ctx, &bars->item_empty[slot], ((n / kItemSlots) & 1) ^ 1, kItemWait);
  if (lane == 0) {
    if (*(volatile int*)&bars->abort) it.last = 1;
    slots[slot] = it;
    mbar_arrive(smem_u32(&bars->item_full[slot]));
    const uint32_t far = mapa(smem_u32(&slots[slot]), 1), far_bar = mapa(smem_u32(&bars->item_full[slot]), 1);
    st_async_v4(far, it.q0, it.nq, it.kv0, it.nkeys, far_bar);
    st_async_v4(far + 16, it.lim0, it.prow, it.head, it.seen[0], far_bar);
    st_async_v4(far + 32, it.seen[1], it.tiles[0], it.tiles[1], it.last, far_bar);
  }
  return __shfl_sync(0xffffffffu, it.last, 0) != 0;
}

// The items of a plan: in a fixed one they are the pair's range of pieces, else
// the first is the pair's own and the next come from a counter all pairs
// share, so that a pair done early takes more.
__device__ __forceinline__ void list_plan(const PrefillArgs& a, const Ctx& ctx, Item* slots, int lane) {
  PrefillHeader* head = a.plan.header;
  const int pairs = gridDim.x / 2, pair = cluster_id_x();
  const int np = head->num_pieces, group = head->group_heads;
  const bool fixed = head->fixed != 0;
  const int items = fixed ? a.plan.first_piece[pair + 1] : np * a.num_heads;
  int i = fixed ? a.plan.first_piece[pair] : pair;
  for (uint32_t n = 0;; ++n) {
    Item it{};
    it.last = 1;
    if (i < items) it = item_at(a, np, group, fixed, i);
    if (hand_item(ctx, slots, lane, n, it)) break;
    int next = 0;
    if (lane == 0 && !fixed) next = atomicAdd(&head->next, 1);
    i = fixed ? i + 1 : pairs + __shfl_sync(0xffffffffu, next, 0);
  }
}

// The items without a plan: the pair's span of all items, or, where none is
// long, every pairs-th.
__device__ __noinline__ void list_direct(const PrefillArgs& a, const Ctx& ctx, Item* slots, int lane) {
  const int pairs = gridDim.x / 2, pair = cluster_id_x();
  int4 seq = make_int4(0, 0, 0, 0);
  int blocks = 0, bad = 0;
  if (lane < a.batch) {
    const int q0 = a.cu_q[lane], q1 = a.cu_q[lane + 1], k0 = a.cu_kv[lane], k1 = a.cu_kv[lane + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.total_q) bad |= 8;     // MLA_DEVERR_BAD_QSL
    if (k0 < 0 || k1 < k0 || k1 > a.total_kv) bad |= 2;    // MLA_DEVERR_BAD_SEQ_LEN
    seq = make_int4(q0, q1 - q0, k0, k1 - k0);
    blocks = bad ? 0 : (q1 - q0 + kPrefillRows - 1) / kPrefillRows;
  }
  int units = 0, longest = 0;
  if (a.spans) {
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
      const int c = prefill_block(seq.x, seq.y, seq.z, seq.w, b * kPrefillRows, a.causal).cost();
      units += c + kPrefillItemUnits;
      longest = max(longest, c);
    }
    if (lane == 0) a.plan.splits[pair].pieces = 0;
  }
  int incl = blocks, uincl = units;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o), u = __shfl_up_sync(0xffffffffu, uincl, o);
    if (lane >= o) incl += n, uincl += u;
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  const int before = incl - blocks, items = bad ? 0 : __shfl_sync(0xffffffffu, incl, 31) * a.num_heads;
  if (pair == 0 && lane == 0) a.plan.header->status = bad;

  const bool spans = longest > kPrefillMinChunk && items > 0;
  const unsigned filled = __ballot_sync(0xffffffffu, blocks > 0);
  Span span{};
  int length = 0, used = 1;
  if (spans) {
    const int all = __shfl_sync(0xffffffffu, uincl, 31);
    length = all * a.num_heads;               // below kPrefillDirectUnits
    used = prefill_spans(length, items, pairs);
    span.from = (int)((unsigned)length * min(pair, used) / (unsigned)used);
    span.to = (int)((unsigned)length * min(pair + 1, used) / (unsigned)used);
    span.at = length;
    if (span.from < length) {
      span.head = span.from / all;
      const int rem = span.from - span.head * all;
      span.src = __ffs(__ballot_sync(0xffffffffu, rem >= uincl - units && rem < uincl)) - 1;
      span.at = span.head * all + __shfl_sync(0xffffffffu, uincl - units, span.src);
      while (true) {
        const int cost = span_block(a, seq, span).cost(), rows = __shfl_sync(0xffffffffu, seq.y, span.src);
        if (span.at + kPrefillItemUnits + cost > span.from) break;
        span_advance(span, cost, rows, filled);
      }
    }
  }
  int i = pair;
  for (uint32_t n = 0;; ++n, i += pairs) {
    Item it{};
    it.last = 1;
    if (spans)
      span_next(a, seq, span, filled, length, used, pair, it);
    else if (i < items)
      it = item_direct(a, seq, before, blocks, i);
    if (hand_item(ctx, slots, lane, n, it)) break;
  }
}

// The peer's list warp (one thread) arms its barriers for the items sent to it.
__device__ __forceinline__ void await_items(const Ctx& ctx, const Item* slots) {
  Bars* bars = ctx.bars;
  for (uint32_t n = 0;; ++n) {
    const uint32_t slot = n % kItemSlots;
    mbar_expect_tx(smem_u32(&bars->item_full[slot]), sizeof(Item));
    wait_bar<true>(ctx, &bars->item_full[slot], (n / kItemSlots) & 1, kItemWait);
    const bool last = *(volatile const int*)&slots[slot].last != 0;
    mbar_arrive_remote(ctx.lead(&bars->item_empty[slot]));
    if (last || *(volatile int*)&bars->abort) break;
  }
}

// The next item, read by a whole warp; one without work behind the last or after an abort.
__device__ __forceinline__ Item next_item(const Ctx& ctx, const Item* slots, uint32_t& n, int lane) {
  const uint32_t slot = n % kItemSlots;
  wait_bar<true>(ctx, &ctx.bars->item_full[slot], (n / kItemSlots) & 1, kItemWait);
  Item it = slots[slot];
  if (*(volatile int*)&ctx.bars->abort) it.last = 1;
  __syncwarp();
  if (lane == 0) mbar_arrive_remote(ctx.lead(&ctx.bars->item_empty[slot]));
  ++n;
  return it;
}

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two lanes of one f32x2 instruction
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n"
      " mov.b64 {%0, %1}, x;\n}" : "+f"(a0), "+f"(a1) : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& r0, float& r1, float a0, float a1, float b, float c) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %4};\n mov.b64 z, {%5, %5};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}" : "=f"(r0), "=f"(r1) : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Whether the last value tile of an item has rows past its keys inside the
// last 16-key step of the products.  They meet probabilities of zero, but may
// hold anything, so they are cleared.
__device__ __forceinline__ bool has_tail(const Item& it, int tiles) {
  const int left = it.nkeys - (tiles - 1) * kPrefillTile;
  return left < kPrefillTile && (left & 15);
}

// ------------------------------------------------------------------ producer
// The whole warp walks the items; one elected thread loads the CTA's halves.
__device__ __forceinline__ void load_items(const PrefillArgs& a, const Ctx& ctx, const Item* slots, const CUtensorMap* tm_q,
                                           const CUtensorMap* tm_kv, const CUtensorMap* tm_pe, uint32_t q_smem,
                                           uint32_t ring, int lane) {
  Bars* bars = ctx.bars;
  uint32_t n = 0, items = 0, q_used[2] = {0, 0};
  volatile int* abort_flag = &bars->abort;
  auto query = [&](const Item& it, int t) {
    if (it.tiles[t] == 0 || (t == 1 && narrow_item(it))) return;
    wait_bar(ctx, &bars->q_empty[t], (q_used[t] & 1) ^ 1);
    if (*abort_flag) return;
    if (elect_one()) {
      const uint32_t full = ctx.lead(&bars->q_full[t]);
      mbar_expect_tx_remote(full, kQTile);
#pragma unroll
      for (int c = 0; c < 3; ++c)
        tma_load_3d_pair(q_smem + t * kQTile + c * kQChunk, tm_q, 64 * c, it.head,
                         it.q0 + 256 * t + 128 * (int)ctx.rank, full);
    }
    __syncwarp();
    ++q_used[t];
  };
  while (true) {
    const Item it = next_item(ctx, slots, items, lane);
    if (it.last) break;
    const int tiles = tiles_of(it);
    query(it, 0);
    for (int j = 0; j < tiles; ++j, ++n) {
      const uint32_t stage = n % kStages, parity = ((n / kStages) & 1) ^ 1;
      const uint32_t dst = ring + stage * kStage;
      const int row = it.kv0 + j * kPrefillTile, half = row + 64 * (int)ctx.rank;
      wait_bar(ctx, &bars->k_empty[stage], parity);
      if (*abort_flag) break;
      // test aid: without these keys the waits of the pair run out
      const bool skip = a.debug_skip_tile && blockIdx.x == 0 && n == 0;
      if (!skip && elect_one()) {
        const uint32_t full = ctx.lead(&bars->k_full[stage]);
        mbar_expect_tx_remote(full, kKeyBytes);
        tma_load_3d_pair(dst, tm_kv, 0, it.head, half, full);
        tma_load_3d_pair(dst + kBox, tm_kv, 64, it.head, half, full);
        tma_load_2d_pair(dst + 2 * kBox, tm_pe, 0, half, full);
      }
      __syncwarp();
      if (j == 0) query(it, 1);
      wait_bar(ctx, &bars->v_empty[stage], parity);
      if (*abort_flag) break;
      const bool tail = j + 1 == tiles && has_tail(it, tiles);
      if (elect_one()) {
        // a tile with rows to clear lands on the CTA's own barrier; the
        // clearing warp reports it to the leading CTA
        const uint32_t full = tail ? mapa(smem_u32(&bars->v_tail[stage]), ctx.rank) : ctx.lead(&bars->v_full[stage]);
        const int x = kNope + 64 * (int)ctx.rank;
        mbar_expect_tx_remote(full, kValueBytes);
        tma_load_3d_pair(dst + kKeyBytes, tm_kv, x, it.head, row, full);
        tma_load_3d_pair(dst + kKeyBytes + kBox, tm_kv, x, it.head, row + 64, full);
      }
      __syncwarp();
    }
    if (*abort_flag) break;
  }
  // Every load has landed before the pair ends: the leading CTA's barriers
  // say so for both CTAs, and the pair ends together.
  if (ctx.rank == 0) {
    for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k) {
      wait_bar(ctx, &bars->k_full[k % kStages], (k / kStages) & 1);
      wait_bar(ctx, &bars->v_full[k % kStages], (k / kStages) & 1);
    }
    for (int t = 0; t < 2; ++t)
      if (q_used[t] > 0) wait_bar(ctx, &bars->q_full[t], (q_used[t] - 1) & 1);
  }
}

// ------------------------------------------------------------ clearing warp
__device__ __forceinline__ void clear_tails(const Ctx& ctx, const Item* slots, uint8_t* ring, int lane) {
  Bars* bars = ctx.bars;
  uint32_t n = 0, items = 0, used = 0;     // bit s of `used`: parity of stage s's tail barrier
  while (true) {
    const Item it = next_item(ctx, slots, items, lane);
    if (it.last) break;
    const int tiles = tiles_of(it);
    n += tiles;
    if (tiles == 0 || !has_tail(it, tiles)) continue;
    const uint32_t stage = (n - 1) % kStages;
    wait_bar(ctx, &bars->v_tail[stage], (used >> stage) & 1, kItemWait);   // from the item's start to its last keys
    used ^= 1u << stage;
    const int left = it.nkeys - (tiles - 1) * kPrefillTile, rows = 16 - (left & 15);
    uint8_t* v = ring + stage * kStage + kKeyBytes + left * 128;
    for (int e = lane; e < rows * 8; e += 32) *reinterpret_cast<uint4*>(v + 16 * e) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_release_cluster(ctx.lead(&bars->v_full[stage]));
  }
}

// -------------------------------------------------------------- MMA issuer
// One warp of the leading CTA walks the items; one elected thread issues.
__device__ __forceinline__ void issue_items(const Ctx& ctx, const Item* slots, uint32_t tbase, uint32_t q_smem,
                                            uint32_t ring, int lane) {
  Bars* bars = ctx.bars;
  constexpr uint32_t id_s = idesc_bf16_f32(256, 128, 0, 0);   // K-major queries and keys
  constexpr uint32_t id_o = idesc_bf16_f32(256, 128, 0, 1);   // MN-major values
  constexpr uint32_t hi = desc_hi(1024, kSwizzle128B);
  const uint32_t q_lo = desc_lo(q_smem, 16), k_lo = desc_lo(ring, 16), v_lo = desc_lo(ring + kKeyBytes, kValueBytes);
  uint32_t n = 0, items = 0;               // tiles before, items
  uint32_t q_parity = 0, p_parity = 0;     // bit t: of query tile t's next load, of tile t's next probabilities

  while (true) {
    const Item it = next_item(ctx, slots, items, lane);
    if (it.last) break;
    const bool narrow = narrow_item(it);
    const int tiles = tiles_of(it), steps = max(it.tiles[0], it.tiles[1]);
    const bool tail = tiles > 0 && has_tail(it, tiles);
    // Step i of the two tiles in turn: outputs of key tile i, scores of the
    // next; step -1 has the first scores alone.  One copy of the code (see
    // above): both tiles and all steps run through it.
    for (int i = steps > 0 ? -1 : 0; i < steps; ++i) {
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int count = t ? it.tiles[1] : it.tiles[0];
        if (i >= count || count == 0) continue;
        const int tq = narrow ? 0 : t;
        const bool sole = narrow || t == 1;   // a key tile's last user: tile 1 sees no fewer keys than tile 0
        const uint32_t s_col = tbase + kColS + 128 * t;
        if (i >= 0) {
          const int j = key_tile(narrow, t, i);
          const uint32_t m = n + j, stage = m % kStages;
          const int products = min(kPrefillTile / 16, ((t ? it.seen[1] : it.seen[0]) - j * kPrefillTile + 15) / 16);
          wait_bar(ctx, &bars->v_full[stage], (m / kStages) & 1);
          if (tail && j + 1 == tiles) fence_cluster();   // rows that a thread of each CTA has cleared
          wait_bar(ctx, &bars->p_full[t], (p_parity >> t) & 1);
          p_parity ^= 1u << t;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t v0 = v_lo + stage * (kStage >> 4);
#pragma unroll
            for (int k = 0; k < kPrefillTile / 16; ++k)
              if (k < products)
                mma_pair_ts(tbase + kColO + 128 * t, s_col + 8 * k, v0 + 128 * k, hi, id_o, (i | k) ? 1u : 0u);
            if (sole) mma_commit_pair(smem_u32(&bars->v_empty[stage]));
            if (i + 1 == count) mma_commit_pair(smem_u32(&bars->o_full[t]));
          }
          __syncwarp();
          if (i + 1 == count) continue;
        } else if (t == 0 || !narrow) {
          wait_bar(ctx, &bars->q_full[t], (q_parity >> t) & 1);
          q_parity ^= 1u << t;
        }
        const int j = key_tile(narrow, t, i + 1);
        const uint32_t m = n + j, stage = m % kStages;
        wait_bar(ctx, &bars->k_full[stage], (m / kStages) & 1);
        tc_fence_after();
        if (elect_one()) {
          const uint32_t k0 = k_lo + stage * (kStage >> 4), q0 = q_lo + tq * (kQTile >> 4);
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_pair_ss(s_col, q0 + ((c * kQChunk) >> 4) + 2 * k, hi, k0 + ((c * kBox) >> 4) + 2 * k, hi, id_s,
                          (c | k) ? 1u : 0u);
          mma_commit_pair(smem_u32(&bars->s_full[t]));
          if (sole) mma_commit_pair(smem_u32(&bars->k_empty[stage]));
          if (narrow ? j + 1 == tiles : i + 2 == count) mma_commit_pair(smem_u32(&bars->q_empty[tq]));
        }
        __syncwarp();
      }
    }
    n += tiles;
  }
  if (elect_one()) mma_commit_pair(smem_u32(&bars->drain));
  __syncwarp();
}

__device__ __forceinline__ void values4(const __nv_bfloat16* at, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(at);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ float dot8(const __nv_bfloat16* a, const __nv_bfloat16* b, float s) {
  const uint4 x = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(b);
  const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), s);
    s = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), s);
  }
  return s;
}

// A row whose output came out not finite although its sum is: a key that the
// row does not see, but rows beside it do, may hold a value that is not finite
// (0 * inf in the matrix product).  If one of the masked keys [sees, covered)
// does, the warp computes the row again from the keys it sees, with the
// row's own reference and sum; otherwise the result stands.  Only inputs
// with infinities or NaN come here.
__device__ __noinline__ void mend_row(const PrefillArgs& a, int row, int head, int kv0, int sees, int covered,
                                      float ref, float inv, float* part, __nv_bfloat16* out) {
  const int lane = threadIdx.x & 31;
  const __nv_bfloat16* kv = static_cast<const __nv_bfloat16*>(a.kv) + (int64_t)head * a.kv_head_stride;
  bool found = false;
#pragma unroll 4
  for (int j = sees; j < covered; ++j) {
    float v[4];
    values4(kv + (int64_t)(kv0 + j) * a.kv_token_stride + kNope + 4 * lane, v);
    for (int e = 0; e < 4; ++e) found |= !(fabsf(v[e]) < INFINITY);
  }
  if (!__any_sync(0xffffffffu, found)) return;
  const __nv_bfloat16* q =
      static_cast<const __nv_bfloat16*>(a.q) + (int64_t)row * a.q_token_stride + (int64_t)head * a.q_head_stride;
  const __nv_bfloat16* pe = static_cast<const __nv_bfloat16*>(a.k_pe);
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int j0 = 0; j0 < sees; j0 += 32) {
    float p = 0.f;
    if (j0 + lane < sees) {
      const __nv_bfloat16* k = kv + (int64_t)(kv0 + j0 + lane) * a.kv_token_stride;
      const __nv_bfloat16* r = pe + (int64_t)(kv0 + j0 + lane) * a.k_pe_stride;
      float s = 0.f;
#pragma unroll 8
      for (int d = 0; d < kNope; d += 8) s = dot8(q + d, k + d, s);
#pragma unroll
      for (int d = 0; d < 64; d += 8) s = dot8(q + kNope + d, r + d, s);
      p = fast_exp2(fmaf(s, a.scale_log2, -ref));
    }
    const int n = min(32, sees - j0);
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      float v[4];
      values4(kv + (int64_t)(kv0 + j0 + j) * a.kv_token_stride + kNope + 4 * lane, v);
      for (int e = 0; e < 4; ++e) o[e] = fmaf(pj, v[e], o[e]);
    }
  }
  for (int e = 0; e < 4; ++e) {
    if (part)
      part[4 * lane + e] = o[e] * inv;
    else
      out[4 * lane + e] = __float2bfloat16_rn(o[e] * inv);
  }
}

// The pieces below that a tile or an item runs once are kept as small loops:
// fetching straight-line code for them cost several thousand cycles each time
// (the tile's own code is the only part that is hot).

// Scores of keys that a row does not see, the tile's from `left` on, become -inf.
// The warp's rows see `fewest` of its keys or more and none behind `most`.
__device__ __forceinline__ void mask_tile(uint32_t s_col, int left, int fewest, int most) {
  const int g0 = max(fewest, 0) >> 5;
  left -= 32 * g0;
#pragma unroll 1
  for (int g = g0; g < 4 && 32 * g < most; ++g, left -= 32) {
    uint32_t s[32];
    tmem_ld32(s_col + 32 * g, s);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; ++c) s[c] = c < left ? s[c] : 0xff800000u;
    tmem_st32(s_col + 32 * g, s);
  }
  uint32_t none[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) none[c] = 0xff800000u;
#pragma unroll 1
  for (int g = 2 * ((most + 31) >> 5); g < 8; ++g) tmem_st16(s_col + 16 * g, none);
  tmem_wait_st();
}

// One tile of a warp's rows: scores to probabilities, with the row's reference and sum.
__device__ __forceinline__ void softmax_tile(uint32_t s_col, uint32_t o_col, float scale, bool first, float& ref,
                                             float& sum) {
  uint32_t s[4][32];
  float top[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) tmem_ld32_max(s_col + 32 * g, s[g], top[g]);
  tmem_wait_ld();
  float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  m *= scale;
  const bool raise = m > ref + kRescale;
  if (__any_sync(0xffffffffu, raise)) {
    const float next = raise ? m : ref;
    const float alpha = raise ? fast_exp2(ref - next) : 1.f;   // ref = -inf: 0
    if (!first) {
      // the scores' arrival implies that the products before them are
      // done, and the next one waits for this warp
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        uint32_t o[16];
        tmem_ld16(o_col + 16 * g, o);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
        tmem_st16(o_col + 16 * g, o);
      }
    }
    sum *= alpha;
    ref = next;
  }
  const float sub = ref == -INFINITY ? 0.f : ref;
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t p[16];
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      float x0, x1, x2, x3;
      fma2(x0, x1, __uint_as_float(s[g][c]), __uint_as_float(s[g][c + 1]), scale, -sub);
      fma2(x2, x3, __uint_as_float(s[g][c + 2]), __uint_as_float(s[g][c + 3]), scale, -sub);
      x0 = fast_exp2(x0), x1 = fast_exp2(x1), x2 = fast_exp2(x2), x3 = fast_exp2(x3);
      add2(s0, s1, x0, x1);
      add2(s2, s3, x2, x3);
      p[c / 2] = pack_bf16x2(x0, x1);
      p[c / 2 + 1] = pack_bf16x2(x2, x3);
    }
    tmem_st16(s_col + 16 * g, p);
  }
  sum += (s0 + s1) + (s2 + s3);
}

// ------------------------------------------------------------------ softmax
__device__ __forceinline__ void softmax_items(const PrefillArgs& a, const Ctx& ctx, const Item* slots, float2* handover,
                                              uint32_t tbase, int warp, int lane) {
  Bars* bars = ctx.bars;
  const int t = warp >> 2, quad = warp & 3;
  const uint32_t lanes = (uint32_t)(32 * quad) << 16;
  const uint32_t s_col = tbase + lanes + kColS + 128 * t, o_col = tbase + lanes + kColO + 128 * t;
  const float scale = a.scale_log2;
  const uint32_t p_full = ctx.lead(&bars->p_full[t]);
  uint32_t items = 0, s_used = 0, o_used[2] = {0, 0}, handed = 0;

  while (true) {
    const Item it = next_item(ctx, slots, items, lane);
    if (it.last) break;
    const bool narrow = narrow_item(it);
    const int tiles = it.tiles[t];
    const int row = (narrow ? 0 : 256 * t) + 128 * (int)ctx.rank + 32 * quad + lane;
    const int sees = min(max(it.lim0 + (a.causal ? row : 0), 0), it.nkeys);
    const int warp_sees = min(max(it.lim0 + (a.causal ? row - lane : 0), 0), it.nkeys);   // its first row: the fewest
    const int warp_most = min(max(it.lim0 + (a.causal ? row - lane + 31 : 0), 0), it.nkeys);   // its last: the most
    const bool idle = row - lane >= it.nq;          // a warp without rows only keeps the others company
    float ref = -INFINITY, sum = 0.f;

    for (int i = 0; i < tiles; ++i, ++s_used) {
      const int j = key_tile(narrow, t, i);
      wait_bar(ctx, &bars->s_full[t], s_used & 1);
      tc_fence_after();
      if (idle || warp_most <= j * kPrefillTile) {
        if (!idle) {
          // every key of the tile is masked
          uint32_t zero[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) zero[c] = 0;
#pragma unroll 1
          for (int g = 0; g < 4; ++g) tmem_st16(s_col + 16 * g, zero);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(p_full);
        continue;
      }
      if (warp_sees < (j + 1) * kPrefillTile) mask_tile(s_col, sees - j * kPrefillTile, warp_sees - j * kPrefillTile, warp_most - j * kPrefillTile);
      softmax_tile(s_col, o_col, scale, i == 0, ref, sum);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(p_full);
    }

    // the item's results
    const bool both = narrow && it.tiles[1] > 0;    // tile 1 holds a part of the same rows
    if (t == 1 && narrow) {
      if (!both) continue;
      ++o_used[1];
      if (idle) continue;
      // the warp of tile 0 with the same rows joins them
      handover[32 * quad + lane] = make_float2(ref, sum);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->x_full[quad]));
      wait_bar(ctx, &bars->x_done[quad], handed & 1);
      ++handed;
      continue;
    }
    for (int u = 0; u < 2; ++u) {
      if (it.tiles[u] == 0) continue;
      if (u == t || both) wait_bar(ctx, &bars->o_full[u], o_used[u] & 1);
      ++o_used[u];
    }
    tc_fence_after();
    if (idle) continue;
    float w0 = 1.f, w1 = 0.f;                       // weights of this tile's and of tile 1's part
    bool some0 = true, some1 = false;               // whether the row sees a key of each (a NaN sum is not 0)
    if (both) {
      wait_bar(ctx, &bars->x_full[quad], handed & 1);
      ++handed;
      const float2 other = handover[32 * quad + lane];
      const float top = fmaxf(ref, other.x), sub = top == -INFINITY ? 0.f : top;
      w0 = fast_exp2(ref - sub);
      w1 = fast_exp2(other.x - sub);
      some0 = sum != 0.f;
      some1 = other.y != 0.f;
      sum = (some0 ? sum * w0 : 0.f) + (some1 ? other.y * w1 : 0.f);
      ref = top;
    }
    const bool live = row < it.nq;
    const bool none = sum == 0.f;                   // no key seen
    const float inv = none ? 0.f : 1.f / sum;
    const float lse = none ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
    w0 *= inv, w1 *= inv;
    const int64_t at = (int64_t)(it.q0 + row) * a.num_heads + it.head;
    const int64_t part_at = (int64_t)it.prow + row;
    float spoilt[4] = {0.f, 0.f, 0.f, 0.f};         // NaN once an output of the row is not finite
    if (live) {
      if (it.prow >= 0)
        a.plan.part_lse[part_at] = lse;
      else if (a.lse)
        a.lse[at] = lse;
    }
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
      uint32_t o[32];
      if (tiles > 0) {
        tmem_ld32(o_col + 32 * g, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) o[c] = none || !some0 ? 0u : __float_as_uint(__uint_as_float(o[c]) * w0);
      if (both) {
        __syncwarp();
        uint32_t e[32];
        tmem_ld32(o_col + 128 + 32 * g, e);
        tmem_wait_ld();
        if (some1)
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(fmaf(__uint_as_float(e[c]), w1, __uint_as_float(o[c])));
      }
#pragma unroll
      for (int c = 0; c < 32; ++c) spoilt[c & 3] = fmaf(__uint_as_float(o[c]), 0.f, spoilt[c & 3]);
      if (live && it.prow >= 0) {
        float* dst = a.plan.part_o + part_at * kNope + 32 * g;
#pragma unroll
        for (int c = 0; c < 4; ++c) st_global_32b(dst + 8 * c, &o[8 * c]);
      } else if (live) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at * kNope + 32 * g;
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = pack_bf16x2(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1]));
        st_global_32b(dst, w);
        st_global_32b(dst + 16, w + 8);
      }
      __syncwarp();
    }
    if (both) {
      tc_fence_before();
      if (lane == 0) mbar_arrive(smem_u32(&bars->x_done[quad]));
    }
    if (a.causal) {
      // keys in the products of this tile that the row does not see
      const int covered = min(it.nkeys, (it.seen[t] + 15) & ~15);
      const bool odd = live && !none && (spoilt[0] + spoilt[1]) + (spoilt[2] + spoilt[3]) != 0.f && fabsf(lse) < INFINITY && sees < covered;
      const unsigned odd_rows = __ballot_sync(0xffffffffu, odd);
      if (odd_rows) count_mending(ctx, lane, 1);
      for (unsigned rows = odd_rows; rows; rows &= rows - 1) {
        const int src = __ffs(rows) - 1;
        const int64_t r_at = __shfl_sync(0xffffffffu, at, src), r_part = __shfl_sync(0xffffffffu, part_at, src);
        mend_row(a, it.q0 + row - lane + src, it.head, it.kv0, __shfl_sync(0xffffffffu, sees, src), covered,
                 __shfl_sync(0xffffffffu, ref, src), __shfl_sync(0xffffffffu, inv, src),
                 it.prow >= 0 ? a.plan.part_o + r_part * kNope : nullptr,
                 static_cast<__nv_bfloat16*>(a.out) + r_at * kNope);
      }
      if (odd_rows) count_mending(ctx, lane, -1);
    }
    tc_fence_before();   // the next item's products may overwrite O once this warp has handed over its P
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                   const __grid_constant__ CUtensorMap tm_pe, const __grid_constant__ PrefillArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* q_smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = q_smem + 2 * kQTile;
  Bars* bars = reinterpret_cast<Bars*>(ring + kStages * kStage);
  Item* slots = reinterpret_cast<Item*>(((uintptr_t)(bars + 1) + 15) & ~(uintptr_t)15);
  float2* handover = reinterpret_cast<float2*>(slots + kItemSlots);   // (reference, sum) of a row of tile 1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&bars->k_full[i]), 2);
      mbar_init(smem_u32(&bars->v_full[i]), 2);
      mbar_init(smem_u32(&bars->k_empty[i]), 1);
      mbar_init(smem_u32(&bars->v_empty[i]), 1);
      mbar_init(smem_u32(&bars->v_tail[i]), 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(smem_u32(&bars->item_full[i]), 1);
      mbar_init(smem_u32(&bars->item_empty[i]), kItemReaders);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bars->q_full[t]), 2);
      mbar_init(smem_u32(&bars->q_empty[t]), 1);
      mbar_init(smem_u32(&bars->s_full[t]), 1);
      mbar_init(smem_u32(&bars->p_full[t]), 8);
      mbar_init(smem_u32(&bars->o_full[t]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bars->x_full[i]), 1);
      mbar_init(smem_u32(&bars->x_done[i]), 1);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    bars->mending = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc_pair(smem_u32(&bars->tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kv);
    tma_prefetch_desc(&tm_pe);
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are initialised before either uses the other's
  tc_fence_after();
  const uint32_t tbase = bars->tmem_base;
  // everything above overlaps the kernel before (the plan)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Ctx ctx{bars, rank, a.wait_limit_ns};

  if (warp < kSoftmaxWarps) {
    setmaxnreg_inc<kRegsSoftmax>();
    softmax_items(a, ctx, slots, handover, tbase, warp, lane);
  } else {
    setmaxnreg_dec<kRegsOther>();
    if (warp == kWarpLoad) {
      load_items(a, ctx, slots, &tm_q, &tm_kv, &tm_pe, smem_u32(q_smem), smem_u32(ring), lane);
    } else if (warp == kWarpMma) {
      if (rank == 0) {
        issue_items(ctx, slots, tbase, smem_u32(q_smem), smem_u32(ring), lane);
        wait_bar(ctx, &bars->drain, 0);   // every product of the pair is done
      }
    } else if (warp == kWarpList) {
      if (rank == 0 && a.direct)
        list_direct(a, ctx, slots, lane);
      else if (rank == 0)
        list_plan(a, ctx, slots, lane);
      else if (lane == 0)
        await_items(ctx, slots);
      __syncwarp();
    } else {
      clear_tails(ctx, slots, ring, lane);
    }
  }
  __syncwarp();
  if (*(volatile int*)&bars->abort) {
    // given up: loads and products in flight finish well within this time
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 1000000ull) {
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // the pair ends together: each reads and signals the other's shared memory
  if (warp == kWarpMma) {
    // The last signal to the peer's own barriers is on its way by now.  Awaited
    // earlier, from the kernel's start, the wait would bound the whole call.
    if (rank == 1) wait_bar(ctx, &bars->drain, 0);
    __syncwarp();
    if (lane == 0) {
      a.plan.header->gave_up[blockIdx.x] = *(volatile int*)&bars->abort;
      if (blockIdx.x == 0) a.plan.header->ctas = gridDim.x;
    }
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

}  // namespace

cudaError_t launch_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const CUtensorMap& tm_pe,
                           const PrefillArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(prefill_kernel, kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * a.pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_kernel, tm_q, tm_kv, tm_pe, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace mla
