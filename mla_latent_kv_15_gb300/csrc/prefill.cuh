// Shared definitions of the expanded attention (mla_prefill): the work plan in
// the caller's workspace and the launchers.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace mla {

constexpr int kNope = 128;           // key width without the rotated part, and value width
constexpr int kPrefillRows = 512;    // query rows per block: two 256-row tiles (tcgen05 M of a CTA pair)
constexpr int kPrefillTile = 128;    // keys per tile
constexpr int kPrefillMaxPairs = 80; // upper bound of the grid (one CTA per SM, in pairs)

// block  = up to 512 consecutive query rows of one sequence (the same for every head)
// piece  = a block's keys [kv0, kv0 + nkeys), cut at multiples of a tile
// item   = a piece and a head: what a CTA pair processes
// A call's errors have a word for each writer, all of them stored by every call
// and joined by the host's read: nothing orders the CTAs' stores.
struct PrefillHeader {
  int status;        // OR of mla_device_error bits of the prefix sums
  int num_pieces;
  int num_split;     // blocks cut into more than one piece
  int next;          // items handed out beyond every pair's first
  int fixed;         // 1: the pieces name their heads and the pairs have theirs from first_piece
  int split_rows;    // rows x heads of the split blocks
  int group_heads;   // heads whose items are interleaved
  int ctas;          // grid of the attention kernel
  int gave_up[2 * kPrefillMaxPairs];   // by CTA: 1 if a bounded wait ran out
};

struct PrefillPiece {  // 32 bytes
  int q0;              // first query row
  int nq;              // rows (<= 512)
  int kv0;             // first key row
  int nkeys;           // keys
  int lim0;            // keys of the piece that row 0 sees (not clamped): row r sees lim0 + r (causal) or lim0
  int prow;            // first partial row (of head 0 where the piece is every head's), or -1: the only piece
  int head;            // the piece's head (fixed plan)
  int pad;
};
static_assert(sizeof(PrefillPiece) == 32, "one aligned 32-byte record");

struct PrefillSplit {  // a block to be joined
  int q0, nq, pieces;
  int head0, heads;    // the heads it is cut for
  int prow;            // partial row of (piece p, head head0 + h, row r): prow + p * stride + h * nq + r
  int before;          // rows * heads of the records before it (with a plan)
  int stride;          // partial rows from a piece to the next
};

struct PrefillPlan {
  PrefillHeader* header;
  int* first_block;      // [batch + 1] blocks before each sequence
  int* first_piece;      // [pairs + 1] fixed plan: first piece of each pair
  PrefillPiece* pieces;
  PrefillSplit* splits;
  float* part_o;         // [max_part_rows][128]
  float* part_lse;       // [max_part_rows]
  int max_pieces;
  int max_part_rows;
};

struct PrefillLayout {
  size_t first_block, first_piece, pieces, splits, part_o, part_lse, total;
  long long max_pieces, max_part_rows;
};

// A fixed plan is made for fewer items (blocks x heads) than this many a pair.
constexpr int kPrefillFixedItems = 8;

// Partial rows of a piece where the pairs cut items by themselves: pair p's
// first piece, of an item that began before it, has those from 2 p times this,
// its last, of an item that ends behind it, the next.
__host__ __device__ inline int prefill_span_rows(int total_q) { return total_q < kPrefillRows ? total_q : kPrefillRows; }

// Byte offsets for a shape.  Automatic splitting makes at most two partial
// pieces per pair (prefill_plan_kernel); a forced count cuts every block.
inline PrefillLayout prefill_layout(int batch, int total_q, int num_heads, int max_splits) {
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PrefillLayout L{};
  const long long mb = (long long)total_q / kPrefillRows + batch;
  const long long auto_rows = 2LL * kPrefillMaxPairs * prefill_span_rows(total_q);
  const long long forced_rows = max_splits > 1 ? (long long)total_q * max_splits * num_heads : 0;
  const long long mp = mb * (max_splits > 1 ? max_splits : 1) + (kPrefillFixedItems + 2) * kPrefillMaxPairs;
  L.max_pieces = mp;
  L.max_part_rows = auto_rows > forced_rows ? auto_rows : forced_rows;
  size_t off = up(sizeof(PrefillHeader));
  L.first_block = off;  off = up(off + sizeof(int) * ((size_t)batch + 1));
  L.first_piece = off;  off = up(off + sizeof(int) * (kPrefillMaxPairs + 1));
  L.pieces = off;       off = up(off + sizeof(PrefillPiece) * (size_t)mp);
  L.splits = off;       off = up(off + sizeof(PrefillSplit) * (size_t)(mb + kPrefillMaxPairs));
  L.part_o = off;       off = up(off + sizeof(float) * kNope * (size_t)L.max_part_rows);
  L.part_lse = off;     off = up(off + sizeof(float) * (size_t)L.max_part_rows);
  L.total = off;
  return L;
}

inline PrefillPlan prefill_plan_from(void* ws, const PrefillLayout& L) {
  char* p = static_cast<char*>(ws);
  return PrefillPlan{reinterpret_cast<PrefillHeader*>(p),
                     reinterpret_cast<int*>(p + L.first_block),
                     reinterpret_cast<int*>(p + L.first_piece),
                     reinterpret_cast<PrefillPiece*>(p + L.pieces),
                     reinterpret_cast<PrefillSplit*>(p + L.splits),
                     reinterpret_cast<float*>(p + L.part_o),
                     reinterpret_cast<float*>(p + L.part_lse),
                     (int)L.max_pieces,
                     (int)L.max_part_rows};
}

struct PrefillArgs {
  // the tensors the maps describe (elements strides), for the rows that are mended one by one
  const void* q;
  int64_t q_token_stride, q_head_stride;
  const void* kv;
  int64_t kv_token_stride, kv_head_stride;
  const void* k_pe;
  int64_t k_pe_stride;
  const int32_t* cu_q;
  const int32_t* cu_kv;
  int batch, total_q, total_kv, num_heads;
  int causal;
  int num_splits;        // 0: automatic
  int direct;            // no plan: the pairs find their items by themselves
  int spans;             // ... which may be cut (then the join is launched)
  int group_heads;       // heads whose keys and values stay in L2 together
  int pairs;             // grid of the attention kernel, in CTA pairs
  float scale_log2;      // scale * log2(e), > 0
  void* out;             // bf16 [total_q, heads, 128]
  float* lse;            // [total_q, heads] or null
  unsigned long long wait_limit_ns;
  int debug_skip_tile;   // test aid: the first pair's leading CTA never loads its first keys
  PrefillPlan plan;
};

// Calls of at most this many sequences need no plan where they have few items
// (below) or no more than this many key rows: every pair's list warp finds its
// items from the prefix sums, a lane a sequence (8 single tokens over up to 8191
// keys: 16 heads 60.2 us a call with the plan, 55.1 without, 1 head 26.5 and
// 22.0, before its spans were shortened).  Over few key rows no item is long enough to be cut or to be taken
// early, and the attention is the only launch (37-token prompt of 16 heads:
// 14 us a call with all three, 11 alone).
constexpr int kPrefillDirectBatch = 32;
constexpr int kPrefillDirectKeys = 512;
constexpr int kPrefillDirectUnits = 1 << 25;   // ... and units of all items (times the pairs they count in 32 bits)

// Costs of items, in units (see the plan): a tile of 128 keys is two, or one
// for a block of up to 256 rows; an item's start and end as much as 3.
constexpr int kPrefillMinChunk = 8, kPrefillMinSpan = 3;
constexpr int kPrefillItemUnits = 3;

#ifdef __CUDACC__
// Query rows r0.. of a sequence of sq rows from q0 over sk keys from k0, as a block.
struct PrefillBlock {
  int q0, nq, kv0, nkeys, lim0;
  __device__ int tiles() const { return (nkeys + kPrefillTile - 1) / kPrefillTile; }
  __device__ int unit() const { return nq > kPrefillRows / 2 ? 2 : 1; }
  __device__ int cost() const { return tiles() * unit(); }
};
// Items laid end to end, each with its fixed cost in front, are cut into
// equal spans: how many, no more than leave each an item's start and
// kPrefillMinSpan units (8 single tokens of one head: 18.4 us with 3, 19.2 with
// 5, 20.8 with 8; a chunk of 600 rows over 4000 keys, 4 heads: 20.2, 21.5, 22.7).
template <class T>
__device__ __forceinline__ int prefill_spans(T length, int items, int pairs) {
  return (int)min((T)pairs, max((T)items, length / (kPrefillItemUnits + kPrefillMinSpan)));
}
// Tiles of an item at `s` that lie before `border`.
template <class T>
__device__ __forceinline__ int prefill_tiles_before(T border, T s, int unit, int tiles) {
  return (int)min(max(border - s - kPrefillItemUnits, (T)0) >> (unit - 1), (T)tiles);
}
__device__ __forceinline__ PrefillBlock prefill_block(int q0, int sq, int k0, int sk, int r0, int causal) {
  PrefillBlock b;
  b.q0 = q0 + r0;
  b.nq = min(kPrefillRows, sq - r0);
  b.kv0 = k0;
  b.lim0 = causal ? sk - sq + 1 + r0 : sk;
  b.nkeys = causal ? min(max(b.lim0 + b.nq - 1, 0), sk) : sk;
  return b;
}
#endif

cudaError_t launch_prefill_plan(const PrefillArgs& a, cudaStream_t s);
// tm_q: {192, heads, total_q} boxes 64 x 1 x 128; tm_kv: {256, heads, total_kv}
// boxes 64 x 1 x 64; tm_pe: {64, total_kv} boxes 64 x 64; all 128-byte swizzled
cudaError_t launch_prefill(const CUtensorMap& tm_q, const CUtensorMap& tm_kv, const CUtensorMap& tm_pe,
                           const PrefillArgs& a, cudaStream_t s);
cudaError_t launch_prefill_combine(const PrefillArgs& a, cudaStream_t s);

}  // namespace mla
