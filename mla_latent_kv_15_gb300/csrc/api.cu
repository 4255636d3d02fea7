// C-ABI entry points of libmla.so (declared in include/mla.h): host-side
// argument validation, TMA descriptor encoding and kernel launches.  Nothing
// here allocates device memory; every buffer belongs to the caller.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <numeric>
#include <string>

#include "../../include/mla.h"
#include "common.cuh"
#include "prefill.cuh"
#include "tmap.cuh"

namespace {

thread_local std::string g_last_error;
thread_local cudaEvent_t g_timing_start = nullptr, g_timing_stop = nullptr;
// bounded-wait test settings of the calling thread (mla_set_decode_wait_test)
thread_local int g_test_skip_tile = 0;
thread_local unsigned long long g_wait_limit_ns = 1000000000ull;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

int ok() {
  g_last_error.clear();
  return MLA_OK;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(MLA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  return n;
}

bool valid_page_size(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

}  // namespace

namespace mla {
// Lets entry points defined in other translation units report an error
// through mla_last_error().
int report_error(int code, const char* msg) { return fail(code, "%s", msg); }
}  // namespace mla

namespace {

// Checks of a cache write's arguments (mla_cache_write, mla_decode_step);
// fills *w when they pass (num_tokens == 0 passes and writes nothing).
int cache_write_args(const void* kv_c, const void* k_pe, const int64_t* slot_mapping, int64_t num_tokens, void* cache,
                     int64_t num_blocks, int page_size, int cache_dtype, float kv_scale, mla::CacheWriteArgs* w) {
  if (num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %lld)", (long long)num_tokens);
  if (cache_dtype != MLA_BF16 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_INVALID_ARG, "cache_dtype must be MLA_BF16 or MLA_FP8_E4M3 (got %d)", cache_dtype);
  if (page_size <= 0 || num_blocks <= 0)
    return fail(MLA_ERR_INVALID_ARG, "page_size and num_blocks must be positive");
  if (cache_dtype == MLA_FP8_E4M3 && !(std::isfinite(kv_scale) && kv_scale > 0.f))
    return fail(MLA_ERR_INVALID_ARG, "kv_scale must be finite and > 0 for an fp8 cache");
  *w = mla::CacheWriteArgs{kv_c, k_pe, slot_mapping, num_tokens, cache, num_blocks * page_size, kv_scale,
                           cache_dtype == MLA_FP8_E4M3};
  if (num_tokens == 0) return ok();
  if (!kv_c || !k_pe || !slot_mapping || !cache) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(kv_c, 16) || !aligned(k_pe, 16) || !aligned(cache, 16) || !aligned(slot_mapping, 8))
    return fail(MLA_ERR_INVALID_ARG, "kv_c, k_pe and cache must be 16-byte aligned, slot_mapping 8-byte aligned");
  return ok();
}

}  // namespace

extern "C" {

const char* mla_last_error(void) { return g_last_error.c_str(); }

int mla_set_decode_timing_events(void* start, void* stop) {
  g_timing_start = start && stop ? static_cast<cudaEvent_t>(start) : nullptr;
  g_timing_stop = start && stop ? static_cast<cudaEvent_t>(stop) : nullptr;
  return ok();
}

int mla_set_decode_wait_test(int skip_first_tile, unsigned long long wait_limit_ns) {
  if (wait_limit_ns == 0) wait_limit_ns = 1000000000ull;
  if (wait_limit_ns < 100000ull || wait_limit_ns > 1000000000ull)
    return fail(MLA_ERR_INVALID_ARG, "wait_limit_ns must be 0 (default 1 s) or in [1e5, 1e9]");
  g_test_skip_tile = skip_first_tile != 0;
  g_wait_limit_ns = wait_limit_ns;
  return ok();
}

int mla_device_sm_count(void) {
  int n = sm_count();
  if (n <= 0) return fail(MLA_ERR_CUDA, "cannot query the current device");
  return n;
}

int mla_cache_write(const void* kv_c, const void* k_pe, const int64_t* slot_mapping, int64_t num_tokens,
                    void* cache, int64_t num_blocks, int page_size, int cache_dtype, float kv_scale,
                    void* stream) {
  mla::CacheWriteArgs w;
  const int rc = cache_write_args(kv_c, k_pe, slot_mapping, num_tokens, cache, num_blocks, page_size, cache_dtype,
                                  kv_scale, &w);
  if (rc != MLA_OK || num_tokens == 0) return rc;
  cudaError_t e = mla::launch_cache_write(w, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "cache write launch");
  return ok();
}

size_t mla_decode_workspace_size(int batch, int total_q, int num_heads, int max_splits) {
  if (batch <= 0 || total_q <= 0 || num_heads <= 0 || max_splits < 0) return 0;
  return mla::workspace_layout(batch, total_q, num_heads, max_splits).total;
}

}  // extern "C"

namespace {

// The decode of mla_decode (q8 == nullptr: bf16 q_abs and q_pe), of
// mla_decode_fp8q (q8: e4m3 [q_abs | q_pe] rows with q_scale, e4m3 cache) and
// of mla_decode_shared (shared: the prefixes, with their block table).
int decode_impl(const void* q_abs, const void* q_pe, const void* q8, float q_scale, const void* cache,
                int64_t num_blocks, int page_size, int cache_dtype, float kv_scale, const int32_t* block_table,
                int max_pages_per_seq, const int32_t* seq_lens, int batch, const int32_t* query_start_loc,
                int total_q, int num_heads, float scale, int num_splits, void* out, float* lse, void* workspace,
                size_t workspace_bytes, void* stream, const mla::CacheWriteArgs* write = nullptr,
                const mla::QuantArgs* quant = nullptr, const mla::SharedArgs* shared = nullptr,
                const int32_t* prefix_table = nullptr) {
  if (batch < 0 || total_q < 0) return fail(MLA_ERR_INVALID_ARG, "batch and total_q must be >= 0");
  if (num_heads < 1 || num_heads > 1024) return fail(MLA_ERR_INVALID_ARG, "num_heads must be in [1, 1024]");
  if (batch == 0 || total_q == 0) return ok();
  if (!query_start_loc && total_q != batch)
    return fail(MLA_ERR_INVALID_ARG, "without query_start_loc every request has one query token (total_q == batch)");
  if ((q8 ? !q8 : (!q_abs || !q_pe)) || !cache || !block_table || !seq_lens || !out || !workspace)
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if ((q8 ? !aligned(q8, 16) : (!aligned(q_abs, 16) || !aligned(q_pe, 16))) || !aligned(cache, 16) ||
      !aligned(out, 16))
    return fail(MLA_ERR_INVALID_ARG, "the query, cache and out must be 16-byte aligned");
  if (q8 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_UNSUPPORTED, "an e4m3 query needs an e4m3 cache");
  if (q8 && !(std::isfinite(q_scale) && q_scale > 0.f))
    return fail(MLA_ERR_INVALID_ARG, "q_scale must be finite and > 0");
  if (q8 && !(std::isnormal(q_scale * kv_scale)))
    return fail(MLA_ERR_INVALID_ARG, "q_scale * kv_scale must be a normal float (the scores' code-product factor)");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || (query_start_loc && !aligned(query_start_loc, 4)) ||
      (lse && !aligned(lse, 4)))
    return fail(MLA_ERR_INVALID_ARG, "block_table, seq_lens, query_start_loc and lse must be 4-byte aligned");
  if (!aligned(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (!valid_page_size(page_size))
    return fail(MLA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256 (got %d)", page_size);
  if (num_blocks <= 0 || num_blocks * (int64_t)page_size >= (int64_t)1 << 31)
    return fail(MLA_ERR_INVALID_ARG, "num_blocks * page_size must be in [1, 2^31)");
  if (max_pages_per_seq <= 0) return fail(MLA_ERR_INVALID_ARG, "max_pages_per_seq must be positive");
  if ((int64_t)total_q * num_heads >= ((int64_t)1 << 31) - 1024)
    return fail(MLA_ERR_INVALID_ARG, "total_q * num_heads must be below 2^31");
  if (cache_dtype != MLA_BF16 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_INVALID_ARG, "cache_dtype must be MLA_BF16 or MLA_FP8_E4M3 (got %d)", cache_dtype);
  if (cache_dtype == MLA_FP8_E4M3 && !(std::isfinite(kv_scale) && kv_scale > 0.f))
    return fail(MLA_ERR_INVALID_ARG, "kv_scale must be finite and > 0 for an fp8 cache");
  if (!std::isfinite(scale) || scale == 0.f) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and nonzero");
  if (num_splits < 0 || num_splits > 4096) return fail(MLA_ERR_INVALID_ARG, "num_splits must be in [0, 4096]");

  const mla::WorkspaceLayout L =
      mla::workspace_layout(batch, total_q, num_heads, num_splits, shared ? shared->prefixes : -1);
  if (workspace_bytes < L.total)
    return fail(MLA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, L.total);
  const int sms = sm_count();
  if (sms < 2) return fail(MLA_ERR_CUDA, "cannot query the current device");
  const int clusters = sms / 2 < mla::kMaxClusters ? sms / 2 : mla::kMaxClusters;

  const uint64_t rows = (uint64_t)total_q * num_heads;
  const uint64_t kv_rows = (uint64_t)num_blocks * page_size;
  // Each CTA of a pair reads latent columns [256r, 256r+256) and rope columns
  // [512+32r, 512+32r+32): tensor maps for the latent boxes and the rope boxes
  // of the query and of the cache.
  CUtensorMap tm_q, tm_qr, tm_kv, tm_kvr;
  const uint32_t kv_box_rows = page_size < mla::kTile ? page_size : mla::kTile;
  bool enc;
  if (q8) {
    // e4m3 query rows and cache rows (576 bytes wide): 128-byte latent boxes
    // (128-B swizzle) and 32-byte rope boxes (32-B swizzle)
    enc = mla::encode_tmap_2d(&tm_q, q8, CU_TENSOR_MAP_DATA_TYPE_UINT8, mla::kDqk, rows, mla::kDqk, 128, 64,
                              CU_TENSOR_MAP_SWIZZLE_128B) &&
          mla::encode_tmap_2d(&tm_qr, q8, CU_TENSOR_MAP_DATA_TYPE_UINT8, mla::kDqk, rows, mla::kDqk, 32, 64,
                              CU_TENSOR_MAP_SWIZZLE_32B) &&
          mla::encode_tmap_2d(&tm_kv, cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, mla::kDqk, kv_rows, mla::kDqk, 128,
                              kv_box_rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
          mla::encode_tmap_2d(&tm_kvr, cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, mla::kDqk, kv_rows, mla::kDqk, 32,
                              kv_box_rows, CU_TENSOR_MAP_SWIZZLE_32B);
  } else {
    // bf16 q_abs (64-dim boxes, 128-B swizzle) and q_pe (32-dim boxes, 64-B swizzle)
    enc = mla::encode_tmap_2d(&tm_q, q_abs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kLkv, rows, mla::kLkv * 2, 64, 64,
                              CU_TENSOR_MAP_SWIZZLE_128B) &&
          mla::encode_tmap_2d(&tm_qr, q_pe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kRope, rows, mla::kRope * 2, 32,
                              64, CU_TENSOR_MAP_SWIZZLE_64B);
    if (cache_dtype == MLA_BF16)
      enc = enc &&
            mla::encode_tmap_2d(&tm_kv, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kDqk, kv_rows, mla::kDqk * 2,
                                64, kv_box_rows, CU_TENSOR_MAP_SWIZZLE_128B) &&
            mla::encode_tmap_2d(&tm_kvr, cache, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kDqk, kv_rows, mla::kDqk * 2,
                                32, kv_box_rows, CU_TENSOR_MAP_SWIZZLE_64B);
    else  // e4m3 codes land unswizzled and are expanded on chip
      enc = enc &&
            mla::encode_tmap_2d(&tm_kv, cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, mla::kDqk, kv_rows, mla::kDqk,
                                shared ? 256 : 64, kv_box_rows, CU_TENSOR_MAP_SWIZZLE_NONE) &&
            mla::encode_tmap_2d(&tm_kvr, cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, mla::kDqk, kv_rows, mla::kDqk, 32,
                                kv_box_rows, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  // the epilogue stores whole 32-row x 64-dim pieces of the output and of the
  // split partials with TMA (128-B swizzle, as they are staged on chip)
  const mla::Plan plan = mla::plan_from_workspace(workspace, L);
  CUtensorMap tm_out, tm_part;
  enc = enc &&
        mla::encode_tmap_2d(&tm_out, out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kLkv, rows, mla::kLkv * 2, 64, 32,
                            CU_TENSOR_MAP_SWIZZLE_128B) &&
        mla::encode_tmap_2d(&tm_part, plan.part_o, CU_TENSOR_MAP_DATA_TYPE_UINT16, mla::kLkv,
                            (uint64_t)L.max_units * mla::kRows, mla::kLkv * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!enc) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor layout");

  mla::DecodeArgs a{};
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.qsl = query_start_loc;
  a.batch = batch;
  a.num_heads = num_heads;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.num_blocks = (int)num_blocks;
  a.total_rows = (int)rows;
  // an e4m3 row holds value / kv_scale: the scale folds into the scores and the output
  const float kvs = cache_dtype == MLA_FP8_E4M3 ? kv_scale : 1.f;
  // the kernel works with a positive scale; a negative one negates q instead
  a.scale_log2 = std::fabs(scale) * 1.4426950408889634f * kvs;
  if (q8) {
    // the e4m3-query kernel turns its code-product sums into real partial
    // scores (x q_scale x kv_scale) before the exchange
    a.qk_scale = q_scale * kv_scale;
    a.scale_log2 = std::fabs(scale) * 1.4426950408889634f;
  }
  a.neg_q = scale < 0.f;
  a.out_scale = kvs;
  a.out = out;
  a.lse = lse;
  a.wait_limit_ns = g_wait_limit_ns;
  a.debug_skip_tile = g_test_skip_tile;
  a.plan = plan;
  a.prefix_table = prefix_table;
  a.max_prefix_pages = shared ? shared->max_pages : 0;

  cudaStream_t s = (cudaStream_t)stream;
  // small head counts with one query token per request (total_q == batch):
  // 32-row groups and the decode variant with small receive buffers and a
  // deeper cache ring.  Groups never outnumber the batch then: a request with
  // Sq tokens gives ceil(Sq * N / 32) <= Sq groups.
  const int small_rows = !shared && !q8 && cache_dtype == MLA_BF16 && num_heads <= 32 && total_q == batch;
  const int variant = q8 ? 3 : (cache_dtype == MLA_FP8_E4M3 ? 1 : (small_rows ? 2 : 0));
  // whether a plan of this call may have long units of many rows (a pair's span of
  // the axis holds no more tiles than its share).  By the tables' width, since the
  // lengths are the device's: 8 requests of 16 heads behind 512 keys take 15.9 us,
  // with tables 32768 keys wide 17.5
  const int long_units =
      shared && rows > 64 &&
      (num_splits > 0 ? std::max(max_pages_per_seq, shared->max_pages) * (int64_t)page_size >= mla::kCodedTiles * mla::kTile
                      : shared->tiles >= (int64_t)mla::kCodedTiles * clusters);
  cudaError_t e = shared ? mla::launch_shared_plan(seq_lens, query_start_loc, batch, num_heads, max_pages_per_seq,
                                                   page_size, num_splits, clusters, a.plan, *shared, s)
                         : mla::launch_plan(seq_lens, query_start_loc, batch, num_heads, max_pages_per_seq, page_size,
                                            num_splits, clusters, small_rows ? 32 : mla::kRows, a.plan, write, quant,
                                            sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "plan launch");
  const bool timed = g_timing_start && g_timing_stop;
  if (timed && (e = cudaEventRecord(g_timing_start, s)) != cudaSuccess) return cuda_fail(e, "timing event");
  e = shared ? mla::launch_decode_shared(tm_q, tm_qr, tm_kv, tm_kvr, tm_out, tm_part, variant, long_units, a, clusters, s)
             : mla::launch_decode(tm_q, tm_qr, tm_kv, tm_kvr, tm_out, tm_part, variant, a, clusters, s);
  if (e != cudaSuccess) return cuda_fail(e, "decode launch");
  if (timed && (e = cudaEventRecord(g_timing_stop, s)) != cudaSuccess) return cuda_fail(e, "timing event");
  e = shared ? mla::launch_combine_shared(a, sms, s) : mla::launch_combine(a, L.max_groups, sms, s);
  if (e != cudaSuccess) return cuda_fail(e, "combine launch");
  return ok();
}

}  // namespace

extern "C" {

int mla_decode(const void* q_abs, const void* q_pe, const void* cache, int64_t num_blocks, int page_size,
               int cache_dtype, float kv_scale, const int32_t* block_table, int max_pages_per_seq,
               const int32_t* seq_lens, int batch, const int32_t* query_start_loc, int total_q, int num_heads,
               float scale, int num_splits, void* out, float* lse, void* workspace, size_t workspace_bytes,
               void* stream) {
  return decode_impl(q_abs, q_pe, nullptr, 0.f, cache, num_blocks, page_size, cache_dtype, kv_scale, block_table,
                     max_pages_per_seq, seq_lens, batch, query_start_loc, total_q, num_heads, scale, num_splits, out,
                     lse, workspace, workspace_bytes, stream);
}

int mla_decode_step(const void* kv_c, const void* k_pe, const int64_t* slot_mapping, int64_t num_new_tokens,
                    const void* q_abs, const void* q_pe, void* cache, int64_t num_blocks, int page_size,
                    int cache_dtype, float kv_scale, const int32_t* block_table, int max_pages_per_seq,
                    const int32_t* seq_lens, int batch, const int32_t* query_start_loc, int total_q, int num_heads,
                    float scale, int num_splits, void* out, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream) {
  mla::CacheWriteArgs w;
  const int rc = cache_write_args(kv_c, k_pe, slot_mapping, num_new_tokens, cache, num_blocks, page_size,
                                  cache_dtype, kv_scale, &w);
  if (rc != MLA_OK) return rc;
  if (batch == 0 || total_q == 0)   // no decode: the write alone
    return mla_cache_write(kv_c, k_pe, slot_mapping, num_new_tokens, cache, num_blocks, page_size, cache_dtype,
                           kv_scale, stream);
  return decode_impl(q_abs, q_pe, nullptr, 0.f, cache, num_blocks, page_size, cache_dtype, kv_scale, block_table,
                     max_pages_per_seq, seq_lens, batch, query_start_loc, total_q, num_heads, scale, num_splits, out,
                     lse, workspace, workspace_bytes, stream, num_new_tokens > 0 ? &w : nullptr);
}

int mla_decode_fp8q_step(const void* kv_c, const void* k_pe, const int64_t* slot_mapping, int64_t num_new_tokens,
                         const void* q_abs, const void* q_pe, float q_scale, void* q_fp8, void* cache,
                         int64_t num_blocks, int page_size, float kv_scale, const int32_t* block_table,
                         int max_pages_per_seq, const int32_t* seq_lens, int batch, const int32_t* query_start_loc,
                         int total_q, int num_heads, float scale, int num_splits, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, void* stream) {
  mla::CacheWriteArgs w;
  int rc = cache_write_args(kv_c, k_pe, slot_mapping, num_new_tokens, cache, num_blocks, page_size, MLA_FP8_E4M3,
                            kv_scale, &w);
  if (rc != MLA_OK) return rc;
  if (batch == 0 || total_q == 0)   // no decode: the write alone
    return mla_cache_write(kv_c, k_pe, slot_mapping, num_new_tokens, cache, num_blocks, page_size, MLA_FP8_E4M3,
                           kv_scale, stream);
  if (!q_abs || !q_pe || !q_fp8) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q_abs, 16) || !aligned(q_pe, 16) || !aligned(q_fp8, 16))
    return fail(MLA_ERR_INVALID_ARG, "q_abs, q_pe and q_fp8 must be 16-byte aligned");
  if (!(std::isfinite(q_scale) && q_scale > 0.f)) return fail(MLA_ERR_INVALID_ARG, "q_scale must be finite and > 0");
  if (total_q < 0 || num_heads < 1 || num_heads > 1024)
    return fail(MLA_ERR_INVALID_ARG, "total_q must be >= 0 and num_heads in [1, 1024]");
  const mla::QuantArgs qa{q_abs, q_pe, (int64_t)total_q * num_heads, q_scale, static_cast<uint8_t*>(q_fp8)};
  return decode_impl(nullptr, nullptr, q_fp8, q_scale, cache, num_blocks, page_size, MLA_FP8_E4M3, kv_scale,
                     block_table, max_pages_per_seq, seq_lens, batch, query_start_loc, total_q, num_heads, scale,
                     num_splits, out, lse, workspace, workspace_bytes, stream, num_new_tokens > 0 ? &w : nullptr,
                     &qa);
}

int mla_decode_fp8q(const void* q_fp8, float q_scale, const void* cache, int64_t num_blocks, int page_size,
                    float kv_scale, const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens,
                    int batch, const int32_t* query_start_loc, int total_q, int num_heads, float scale,
                    int num_splits, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  return decode_impl(nullptr, nullptr, q_fp8, q_scale, cache, num_blocks, page_size, MLA_FP8_E4M3, kv_scale,
                     block_table, max_pages_per_seq, seq_lens, batch, query_start_loc, total_q, num_heads, scale,
                     num_splits, out, lse, workspace, workspace_bytes, stream);
}

int mla_decode_status(const void* workspace, int* status, void* stream) {
  if (!workspace || !status) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaMemcpyAsync(status, workspace, sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  return ok();
}

int mla_merge_states(const void* o_a, const float* lse_a, const void* o_b, const float* lse_b, int64_t rows, int dim,
                     int o_dtype, void* out, float* lse_out, void* stream) {
  if (rows < 0) return fail(MLA_ERR_INVALID_ARG, "rows must be >= 0");
  if (dim <= 0 || dim % 8 != 0 || dim > 4096) return fail(MLA_ERR_INVALID_ARG, "dim must be a multiple of 8 in [8, 4096]");
  if (o_dtype != MLA_BF16 && o_dtype != MLA_FP32)
    return fail(MLA_ERR_INVALID_ARG, "o_dtype must be MLA_BF16 or MLA_FP32 (got %d)", o_dtype);
  if (rows == 0) return ok();
  if (!o_a || !lse_a || !o_b || !lse_b || !out) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(o_a, 16) || !aligned(o_b, 16) || !aligned(out, 16))
    return fail(MLA_ERR_INVALID_ARG, "o_a, o_b and out must be 16-byte aligned");
  if (!aligned(lse_a, 4) || !aligned(lse_b, 4) || (lse_out && !aligned(lse_out, 4)))
    return fail(MLA_ERR_INVALID_ARG, "LSE arrays must be 4-byte aligned");
  if (lse_out && (lse_out == lse_a || lse_out == lse_b))
    return fail(MLA_ERR_INVALID_ARG, "lse_out must not alias lse_a or lse_b");
  const int sms = sm_count();   // of the current device, per call
  if (sms < 1) return fail(MLA_ERR_CUDA, "cannot query the current device");
  cudaError_t e = mla::launch_merge_states(o_a, lse_a, o_b, lse_b, rows, dim, o_dtype == MLA_BF16, out, lse_out,
                                           sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "merge launch");
  return ok();
}

}  // extern "C"

namespace {

// Shared body of the two per-head projections: validation of what both have
// in common, tensor maps, launch.
int head_proj(const char* name, const void* x, int64_t x_stride, const void* w, int64_t T, int N, int d_in,
              int d_out, void* y, void* stream) {
  if (T < 0) return fail(MLA_ERR_INVALID_ARG, "%s: num_tokens must be >= 0", name);
  if (T > 65535LL * 128) return fail(MLA_ERR_UNSUPPORTED, "%s: num_tokens must be <= 8388480", name);
  if (N < 1 || N > 1024) return fail(MLA_ERR_INVALID_ARG, "%s: num_heads must be in [1, 1024]", name);
  if (T == 0) return ok();
  if (!x || !w || !y) return fail(MLA_ERR_INVALID_ARG, "%s: null pointer argument", name);
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16))
    return fail(MLA_ERR_INVALID_ARG, "%s: tensors must be 16-byte aligned", name);
  const uintptr_t xb = reinterpret_cast<uintptr_t>(x), yb = reinterpret_cast<uintptr_t>(y);
  const uintptr_t xe = xb + (uintptr_t)((T * N - 1) * x_stride + d_in) * 2, ye = yb + (uintptr_t)(T * N * d_out) * 2;
  if (xb < ye && yb < xe) return fail(MLA_ERR_INVALID_ARG, "%s: the output must not overlap the input", name);
  CUtensorMap tm_x, tm_w;
  if (!mla::encode_tmap_3d(&tm_x, x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)d_in, (uint64_t)N, (uint64_t)T,
                           (uint64_t)x_stride * 2, (uint64_t)x_stride * 2 * N, 64, 1,
                           (uint32_t)mla::head_proj_x_rows(T),
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
      !mla::encode_tmap_2d(&tm_w, w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)d_out, (uint64_t)N * d_in,
                           (uint64_t)d_out * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return fail(MLA_ERR_CUDA, "%s: tensor map encoding failed", name);
  cudaError_t e = mla::launch_head_proj(tm_x, tm_w, y, T, N, d_in, d_out, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, name);
  return ok();
}

}  // namespace

extern "C" {

int mla_q_absorb(const void* q_nope, int64_t q_row_stride, const void* w_uk_t, int64_t num_tokens, int num_heads,
                 int nope_dim, void* ql_nope, void* stream) {
  if (nope_dim < 64 || nope_dim > 1024 || nope_dim % 64 != 0)
    return fail(MLA_ERR_UNSUPPORTED, "mla_q_absorb: nope_dim must be a multiple of 64 in [64, 1024] (got %d)",
                nope_dim);
  if (q_row_stride < nope_dim || q_row_stride % 8 != 0 || q_row_stride > (1LL << 24))
    return fail(MLA_ERR_INVALID_ARG, "mla_q_absorb: q_row_stride must be >= nope_dim, a multiple of 8 and <= 2^24");
  return head_proj("mla_q_absorb", q_nope, q_row_stride, w_uk_t, num_tokens, num_heads, nope_dim, mla::kLkv,
                   ql_nope, stream);
}

int mla_v_up_proj(const void* o_lat, const void* w_uv, int64_t num_tokens, int num_heads, int v_head_dim, void* out,
                  void* stream) {
  const bool ok_dim = (v_head_dim >= 64 && v_head_dim <= 256 && v_head_dim % 64 == 0) || v_head_dim == 512 ||
                      v_head_dim == 1024;
  if (!ok_dim)
    return fail(MLA_ERR_UNSUPPORTED, "mla_v_up_proj: v_head_dim must be 64, 128, 192, 256, 512 or 1024 (got %d)",
                v_head_dim);
  return head_proj("mla_v_up_proj", o_lat, mla::kLkv, w_uv, num_tokens, num_heads, mla::kLkv, v_head_dim, out,
                   stream);
}

int mla_gather_cache(const void* cache, int64_t num_blocks, int page_size, int cache_dtype, float kv_scale,
                     const int32_t* block_table, int max_pages_per_seq, const int32_t* cu_seq_lens,
                     const int32_t* seq_starts, int batch, void* dst, int64_t num_tokens, int32_t* status,
                     void* stream) {
  if (num_tokens < 0 || batch < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens and batch must be >= 0");
  if (cache_dtype != MLA_BF16 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_INVALID_ARG, "cache_dtype must be MLA_BF16 or MLA_FP8_E4M3 (got %d)", cache_dtype);
  if (num_tokens == 0 || batch == 0) return ok();
  if (page_size < 1 || num_blocks < 1 || max_pages_per_seq < 1)
    return fail(MLA_ERR_INVALID_ARG, "page_size, num_blocks and max_pages_per_seq must be positive");
  if (cache_dtype == MLA_FP8_E4M3 && !(std::isfinite(kv_scale) && kv_scale > 0.f))
    return fail(MLA_ERR_INVALID_ARG, "kv_scale must be finite and > 0 for an fp8 cache");
  if (!cache || !block_table || !cu_seq_lens || !dst) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(cache, 16) || !aligned(dst, 16)) return fail(MLA_ERR_INVALID_ARG, "cache and dst must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(cu_seq_lens, 4) || (seq_starts && !aligned(seq_starts, 4)) ||
      (status && !aligned(status, 4)))
    return fail(MLA_ERR_INVALID_ARG, "block_table, cu_seq_lens, seq_starts and status must be 4-byte aligned");
  cudaError_t e = mla::launch_gather(cache, num_blocks, page_size, cache_dtype == MLA_FP8_E4M3, kv_scale,
                                     block_table, max_pages_per_seq, cu_seq_lens, seq_starts, batch, dst,
                                     num_tokens, status, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "gather launch");
  return ok();
}

int mla_quantize_fp8(const void* x, int64_t x_stride, int64_t rows, int width, float scale, void* out,
                     int64_t out_stride, void* stream) {
  if (rows < 0) return fail(MLA_ERR_INVALID_ARG, "rows must be >= 0");
  if (width <= 0 || width % 8 != 0) return fail(MLA_ERR_INVALID_ARG, "width must be a positive multiple of 8");
  if (x_stride < width || x_stride % 8 != 0 || out_stride < width || out_stride % 8 != 0)
    return fail(MLA_ERR_INVALID_ARG, "strides must be multiples of 8 and at least width");
  if (!(std::isfinite(scale) && scale > 0.f)) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (rows == 0) return ok();
  if (!x || !out) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(x, 16) || !aligned(out, 8)) return fail(MLA_ERR_INVALID_ARG, "x must be 16-byte and out 8-byte aligned");
  cudaError_t e = mla::launch_quantize_fp8(x, x_stride, rows, width, scale, out, out_stride, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "quantize launch");
  return ok();
}

int mla_proj_status(int* status, int clear, void* stream) {
  if (!status) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  int kv = 0;
  cudaError_t e = mla::head_proj_status(status, clear, (cudaStream_t)stream);
  if (e == cudaSuccess) e = mla::kv_proj_status(&kv, clear, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "projection status read");
  *status |= kv;
  return ok();
}

}  // extern "C"

namespace {

// Bytes [lo, hi) of a strided tensor of `n0` x `n1` rows of `width` elements
// (strides in elements); `outer` and `inner` are the strides that lead to more
// than one row.  Where the outer one holds all the inner rows, the tensor is
// columns [0, row) of a pitched one.
struct Extent {
  uintptr_t lo, hi;
  uintptr_t width, outer, inner;
  uintptr_t row, pitch;
};
Extent extent(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t width, int64_t elem_bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  const uintptr_t row = (uintptr_t)(((n1 - 1) * s1 + width) * elem_bytes);
  const uintptr_t outer = (uintptr_t)(s0 * elem_bytes), inner = (uintptr_t)(s1 * elem_bytes);
  return Extent{lo, lo + (uintptr_t)(n0 - 1) * outer + row, (uintptr_t)(width * elem_bytes),
                n0 > 1 ? outer : 0, n1 > 1 ? inner : 0, row, n0 > 1 && row <= outer ? outer : 0};
}
Extent dense(const void* p, int64_t bytes) { return extent(p, 1, 0, 1, 0, bytes, 1); }
// Whether `a` bytes and `b` bytes from two addresses, repeated every `step`, share some.
bool columns_meet(uintptr_t a_lo, uintptr_t a, uintptr_t b_lo, uintptr_t b, uintptr_t step) {
  const uintptr_t d = b_lo >= a_lo ? (b_lo - a_lo) % step : (step - (a_lo - b_lo) % step) % step;
  return !(d >= a && d + b <= step);
}
// Whether two tensors may share bytes (column ranges of the same pitched rows,
// of tokens or of heads, are told apart, other strided layouts by their first
// and last bytes).
bool overlap(const Extent& a, const Extent& b) {
  if (!(a.lo < b.hi && b.lo < a.hi)) return false;
  if (a.pitch && a.pitch == b.pitch && !columns_meet(a.lo, a.row, b.lo, b.row, a.pitch)) return false;
  // every row of both begins a multiple of `step` behind its tensor's first
  const uintptr_t step = std::gcd(std::gcd(a.outer, a.inner), std::gcd(b.outer, b.inner));
  return step == 0 || columns_meet(a.lo, a.width, b.lo, b.width, step);
}

// Whether an output (a null one is none) shares bytes with another or an input.
bool any_overlap(const Extent* outputs, int n_out, const Extent* inputs, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    if (!outputs[i].lo) continue;
    for (int j = 0; j < i; ++j)
      if (outputs[j].lo && overlap(outputs[i], outputs[j])) return true;
    for (int j = 0; j < n_in; ++j)
      if (inputs[j].lo && overlap(outputs[i], inputs[j])) return true;
  }
  return false;
}
// `batch` rows of `len` float32 weights, `stride` elements apart.
Extent weight_extent(const void* p, int64_t batch, int64_t stride, int64_t len) {
  return len > 0 ? extent(p, batch, stride, 1, 0, len, 4) : Extent{};
}

constexpr int kMaxBatch = 1 << 20;
constexpr int64_t kMaxKeys = 1LL << 30;     // keys of a request, as far as a table or a row of weights reaches
constexpr int64_t kMaxStride = 1LL << 32;   // elements
bool valid_stride(int64_t s, int64_t least) { return s >= least && s % 8 == 0 && s <= kMaxStride; }

}  // namespace

extern "C" {

int mla_rope_cache_write(const void* kv_c, int64_t kv_c_stride, const void* k_pe, int64_t k_pe_stride,
                         const void* norm_weight, float norm_eps, const int64_t* positions, const float* cos_sin,
                         int64_t max_positions, int interleaved, const int64_t* slot_mapping, int64_t num_tokens,
                         void* cache, int64_t num_blocks, int page_size, int cache_dtype, float kv_scale,
                         void* latent, int64_t latent_stride, const void* q_pe, int64_t q_token_stride,
                         int64_t q_head_stride, int num_heads, void* q_pe_out, int64_t q_out_token_stride,
                         int64_t q_out_head_stride, int* status, void* stream) {
  if (num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %lld)", (long long)num_tokens);
  if (num_tokens > 65535LL * 128) return fail(MLA_ERR_UNSUPPORTED, "num_tokens must be <= 8388480");
  if (cache_dtype != MLA_BF16 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_INVALID_ARG, "cache_dtype must be MLA_BF16 or MLA_FP8_E4M3 (got %d)", cache_dtype);
  if (page_size <= 0 || num_blocks <= 0 || num_blocks > (1LL << 40) / page_size)
    return fail(MLA_ERR_INVALID_ARG, "page_size and num_blocks must be positive and num_blocks * page_size <= 2^40");
  if (max_positions <= 0) return fail(MLA_ERR_INVALID_ARG, "max_positions must be positive");
  if (cache_dtype == MLA_FP8_E4M3 && !(std::isfinite(kv_scale) && kv_scale > 0.f))
    return fail(MLA_ERR_INVALID_ARG, "kv_scale must be finite and > 0 for an fp8 cache");
  if (norm_weight && !(std::isfinite(norm_eps) && norm_eps >= 0.f))
    return fail(MLA_ERR_INVALID_ARG, "norm_eps must be finite and >= 0");
  if (!q_pe != !q_pe_out) return fail(MLA_ERR_INVALID_ARG, "q_pe and q_pe_out are given together or not at all");
  if (q_pe && (num_heads < 1 || num_heads > 1024)) return fail(MLA_ERR_INVALID_ARG, "num_heads must be in [1, 1024]");
  if (num_tokens == 0) return ok();
  if (!kv_c || !k_pe || !positions || !cos_sin || !slot_mapping || !cache)
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(kv_c, 16) || !aligned(k_pe, 16) || !aligned(cache, 16) || !aligned(cos_sin, 16) ||
      !aligned(norm_weight, 16) || !aligned(latent, 16) || !aligned(q_pe, 16) || !aligned(q_pe_out, 16))
    return fail(MLA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  if (!aligned(positions, 8) || !aligned(slot_mapping, 8) || !aligned(status, 4))
    return fail(MLA_ERR_INVALID_ARG, "positions and slot_mapping must be 8-byte aligned, status 4-byte aligned");
  if (!valid_stride(kv_c_stride, 0) || !valid_stride(k_pe_stride, 0))
    return fail(MLA_ERR_INVALID_ARG, "kv_c_stride and k_pe_stride must be multiples of 8 in [0, 2^32]");
  if (latent && !valid_stride(latent_stride, mla::kDqk))
    return fail(MLA_ERR_INVALID_ARG, "latent_stride must be a multiple of 8 in [576, 2^32]");
  const Extent ec = dense(cache, num_blocks * page_size * mla::kDqk * (cache_dtype == MLA_BF16 ? 2 : 1));
  const Extent ek = extent(kv_c, num_tokens, kv_c_stride, 1, 0, mla::kLkv, 2);
  const Extent ep = extent(k_pe, num_tokens, k_pe_stride, 1, 0, mla::kRope, 2);
  // what every token's rows depend on, and the status word (a table larger
  // than any memory is one of unknown size)
  const int64_t table_rows = max_positions < (1LL << 31) ? max_positions : 1;
  const Extent shared[] = {dense(positions, num_tokens * 8), dense(slot_mapping, num_tokens * 8),
                           dense(cos_sin, table_rows * mla::kRope * 4), dense(norm_weight, mla::kLkv * 2),
                           dense(status, 4)};
  auto overlaps_shared = [&](const Extent& x) {
    for (const Extent& s : shared)
      if (s.lo && overlap(x, s)) return true;
    return false;
  };
  if (overlap(ec, ek) || overlap(ec, ep) || overlaps_shared(ec))
    return fail(MLA_ERR_INVALID_ARG, "the cache must not overlap the inputs");
  Extent el{0, 0};
  if (latent) {
    el = extent(latent, num_tokens, latent_stride, 1, 0, mla::kDqk, 2);
    // in place: the latent rows are the input rows themselves
    const bool same = latent == kv_c && static_cast<const char*>(k_pe) == static_cast<char*>(latent) + 2 * mla::kLkv &&
                      (num_tokens == 1 || (latent_stride == kv_c_stride && latent_stride == k_pe_stride));
    if (overlap(el, ec) || overlaps_shared(el) || (!same && (overlap(el, ek) || overlap(el, ep))))
      return fail(MLA_ERR_INVALID_ARG, "latent must not overlap the cache, nor the inputs unless it is their rows");
  }
  mla::RopeWriteArgs w{kv_c,          kv_c_stride,   k_pe,       k_pe_stride,
                       norm_weight,   norm_eps,      positions,  cos_sin,
                       max_positions, slot_mapping,  num_tokens, cache,
                       num_blocks * page_size, kv_scale, latent, latent_stride,
                       q_pe,          q_token_stride, q_head_stride, q_pe_out,
                       q_out_token_stride, q_out_head_stride, num_heads, status};
  if (q_pe) {
    if (!valid_stride(q_token_stride, 0) || !valid_stride(q_head_stride, 0))
      return fail(MLA_ERR_INVALID_ARG, "q_pe strides must be multiples of 8 in [0, 2^32]");
    // the written rows lie apart: heads inside tokens or tokens inside heads
    if (!valid_stride(q_out_token_stride, mla::kRope) || !valid_stride(q_out_head_stride, mla::kRope) ||
        !(q_out_token_stride >= (num_heads - 1) * q_out_head_stride + mla::kRope || num_tokens == 1 ||
          q_out_head_stride >= (num_tokens - 1) * q_out_token_stride + mla::kRope || num_heads == 1))
      return fail(MLA_ERR_INVALID_ARG, "q_pe_out strides must be multiples of 8 that keep its rows of 64 apart");
    const Extent eq = extent(q_pe, num_tokens, q_token_stride, num_heads, q_head_stride, mla::kRope, 2);
    const Extent eo = extent(q_pe_out, num_tokens, q_out_token_stride, num_heads, q_out_head_stride, mla::kRope, 2);
    const bool same = q_pe == q_pe_out && (num_tokens == 1 || q_token_stride == q_out_token_stride) &&
                      (num_heads == 1 || q_head_stride == q_out_head_stride);
    if ((!same && overlap(eq, eo)) || overlap(eo, ec) || overlap(eo, ek) || overlap(eo, ep) || overlap(eq, ec) ||
        overlaps_shared(eo) || (latent && (overlap(el, eo) || overlap(el, eq))))
      return fail(MLA_ERR_INVALID_ARG, "q_pe_out must be q_pe itself or overlap no other argument");
  }
  cudaError_t e = mla::launch_rope_write(w, cache_dtype == MLA_FP8_E4M3, interleaved != 0, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "rotated cache write launch");
  return ok();
}

int mla_kv_up_proj(const void* latent, int64_t latent_stride, const void* w, int64_t num_tokens, int num_heads,
                   int head_dim, void* kv, void* stream) {
  if (num_tokens < 0) return fail(MLA_ERR_INVALID_ARG, "num_tokens must be >= 0 (got %lld)", (long long)num_tokens);
  if (num_tokens > 65535LL * 128) return fail(MLA_ERR_UNSUPPORTED, "num_tokens must be <= 8388480");
  if (num_heads < 1 || num_heads > 1024) return fail(MLA_ERR_INVALID_ARG, "num_heads must be in [1, 1024]");
  if (head_dim < 8 || head_dim > 2048 || head_dim % 8 != 0)
    return fail(MLA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 in [8, 2048] (got %d)", head_dim);
  if (num_tokens == 0) return ok();
  if (!latent || !w || !kv) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(latent, 16) || !aligned(w, 16) || !aligned(kv, 16))
    return fail(MLA_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  if (!valid_stride(latent_stride, mla::kLkv))
    return fail(MLA_ERR_INVALID_ARG, "latent_stride must be a multiple of 8 in [512, 2^32]");
  const int64_t C = (int64_t)num_heads * head_dim;
  const Extent ek = extent(kv, 1, 0, 1, 0, num_tokens * C, 2);
  if (overlap(ek, extent(latent, num_tokens, latent_stride, 1, 0, mla::kLkv, 2)) ||
      overlap(ek, extent(w, 1, 0, 1, 0, C * mla::kLkv, 2)))
    return fail(MLA_ERR_INVALID_ARG, "kv must not overlap the inputs");
  const int sms = sm_count();
  if (sms < 1) return fail(MLA_ERR_CUDA, "cannot query the current device");
  const mla::KvProjShape p = mla::kv_proj_shape(num_tokens, C, sms);
  CUtensorMap tm_x, tm_w, tm_y;
  if (!mla::encode_tmap_2d(&tm_x, latent, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kLkv, (uint64_t)num_tokens,
                           (uint64_t)latent_stride * 2, 64, (uint32_t)p.xrows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !mla::encode_tmap_2d(&tm_w, w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kLkv, (uint64_t)C, mla::kLkv * 2, 64,
                           (uint32_t)p.wrows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !mla::encode_tmap_2d(&tm_y, kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)C, (uint64_t)num_tokens,
                           (uint64_t)C * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B))
    return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor layout");
  cudaError_t e = mla::launch_kv_proj(tm_x, tm_w, tm_y, kv, num_tokens, C, p, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "key/value projection launch");
  return ok();
}

size_t mla_prefill_workspace_size(int batch, int total_q, int num_heads, int max_splits) {
  if (batch <= 0 || total_q <= 0 || num_heads <= 0 || max_splits < 0) return 0;
  return mla::prefill_layout(batch, total_q, num_heads, max_splits).total;
}

int mla_prefill(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* kv, int64_t kv_token_stride,
                int64_t kv_head_stride, const void* k_pe, int64_t k_pe_stride, const int32_t* cu_q,
                const int32_t* cu_kv, int batch, int total_q, int total_kv, int num_heads, float scale, int causal,
                int num_splits, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || total_q < 0 || total_kv < 0)
    return fail(MLA_ERR_INVALID_ARG, "batch, total_q and total_kv must be >= 0");
  if (num_heads < 1 || num_heads > 1024) return fail(MLA_ERR_INVALID_ARG, "num_heads must be in [1, 1024]");
  if (!std::isfinite(scale * 1.4426950408889634f) || scale <= 0.f)
    return fail(MLA_ERR_INVALID_ARG, "scale must be > 0 and scale * log2(e) finite");
  if (num_splits < 0 || num_splits > 4096) return fail(MLA_ERR_INVALID_ARG, "num_splits must be in [0, 4096]");
  if (batch == 0 || total_q == 0) return ok();
  if (total_kv > (1 << 30) || total_q > (1 << 30))
    return fail(MLA_ERR_UNSUPPORTED, "total_q and total_kv must be <= 2^30");
  if ((int64_t)total_q * num_heads >= ((int64_t)1 << 31) - 1024)
    return fail(MLA_ERR_INVALID_ARG, "total_q * num_heads must be below 2^31");
  if (!q || !cu_q || !cu_kv || !out || !workspace || (total_kv > 0 && (!kv || !k_pe)))
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_pe, 16) || !aligned(out, 32))
    return fail(MLA_ERR_INVALID_ARG, "q, kv and k_pe must be 16-byte aligned, out 32-byte aligned");
  if (!aligned(cu_q, 4) || !aligned(cu_kv, 4) || !aligned(lse, 4))
    return fail(MLA_ERR_INVALID_ARG, "cu_q, cu_kv and lse must be 4-byte aligned");
  if (!aligned(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (!valid_stride(q_token_stride, 8) || !valid_stride(q_head_stride, 8) || !valid_stride(kv_token_stride, 8) ||
      !valid_stride(kv_head_stride, 8) || !valid_stride(k_pe_stride, 8))
    return fail(MLA_ERR_INVALID_ARG, "strides must be multiples of 8 in [8, 2^32]");
  const int qd = mla::kNope + mla::kRope, kvd = 2 * mla::kNope;
  const int64_t rows = (int64_t)total_q * num_heads;
  const Extent eo = dense(out, rows * mla::kNope * 2), es = dense(lse, rows * 4);
  const Extent inputs[] = {extent(q, total_q, q_token_stride, num_heads, q_head_stride, qd, 2),
                           dense(cu_q, (batch + 1LL) * 4), dense(cu_kv, (batch + 1LL) * 4),
                           extent(kv, total_kv, kv_token_stride, num_heads, kv_head_stride, kvd, 2),
                           extent(k_pe, total_kv, k_pe_stride, 1, 0, mla::kRope, 2)};
  const int num_inputs = total_kv > 0 ? 5 : 3;
  auto overlaps_inputs = [&](const Extent& x) {
    for (int i = 0; i < num_inputs; ++i)
      if (overlap(x, inputs[i])) return true;
    return false;
  };
  if (overlaps_inputs(eo)) return fail(MLA_ERR_INVALID_ARG, "out must not overlap the inputs");
  const mla::PrefillLayout L = mla::prefill_layout(batch, total_q, num_heads, num_splits);
  if (L.max_part_rows >= 1LL << 31) return fail(MLA_ERR_UNSUPPORTED, "total_q * num_heads * num_splits must be below 2^31");
  if (L.max_pieces * num_heads >= (1LL << 31) - 4096)
    return fail(MLA_ERR_UNSUPPORTED, "batch * num_heads is too large");
  if (lse && (overlap(es, eo) || overlaps_inputs(es)))
    return fail(MLA_ERR_INVALID_ARG, "lse must not overlap out or the inputs");
  if (workspace_bytes < L.total)
    return fail(MLA_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu required", workspace_bytes, L.total);
  const Extent ew = dense(workspace, (int64_t)L.total);
  if (overlap(ew, eo) || (lse && overlap(ew, es)) || overlaps_inputs(ew))
    return fail(MLA_ERR_INVALID_ARG, "the workspace must not overlap the other arguments");
  const int sms = sm_count();
  if (sms < 2) return fail(MLA_ERR_CUDA, "cannot query the current device");

  CUtensorMap tm_q, tm_kv, tm_pe;
  bool enc = mla::encode_tmap_3d(&tm_q, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)qd, (uint64_t)num_heads,
                                 (uint64_t)total_q, (uint64_t)q_head_stride * 2, (uint64_t)q_token_stride * 2, 64, 1,
                                 mla::kPrefillTile, CU_TENSOR_MAP_SWIZZLE_128B);
  tm_kv = tm_pe = tm_q;   // without a key no tile is loaded
  if (total_kv > 0)
    enc = enc &&
          mla::encode_tmap_3d(&tm_kv, kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (uint64_t)kvd, (uint64_t)num_heads,
                              (uint64_t)total_kv, (uint64_t)kv_head_stride * 2, (uint64_t)kv_token_stride * 2, 64, 1,
                              mla::kPrefillTile / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
          mla::encode_tmap_2d(&tm_pe, k_pe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kRope, (uint64_t)total_kv,
                              (uint64_t)k_pe_stride * 2, 64, mla::kPrefillTile / 2, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!enc) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor layout");

  mla::PrefillArgs a{};
  a.q = q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.kv = kv;
  a.kv_token_stride = kv_token_stride;
  a.kv_head_stride = kv_head_stride;
  a.k_pe = k_pe;
  a.k_pe_stride = k_pe_stride;
  a.cu_q = cu_q;
  a.cu_kv = cu_kv;
  a.batch = batch;
  a.total_q = total_q;
  a.total_kv = total_kv;
  a.num_heads = num_heads;
  a.causal = causal != 0;
  a.num_splits = num_splits;
  // as many heads side by side as keep their keys and values in 48 MB of L2
  const int64_t head_bytes = (int64_t)total_kv * kvd * 2 + 1;
  const int64_t fit = (48LL << 20) / head_bytes;
  a.group_heads = (int)(fit < 1 ? 1 : fit > num_heads ? num_heads : fit);
  a.pairs = sms / 2 < mla::kPrefillMaxPairs ? sms / 2 : mla::kPrefillMaxPairs;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out = out;
  a.lse = lse;
  a.wait_limit_ns = g_wait_limit_ns;
  a.debug_skip_tile = g_test_skip_tile;
  a.plan = mla::prefill_plan_from(workspace, L);
  cudaStream_t s = (cudaStream_t)stream;
  // without a plan: few key rows, or few items of not too many units
  const int64_t blocks = (int64_t)total_q / mla::kPrefillRows + batch;
  const bool small = num_splits <= 1 && total_kv <= mla::kPrefillDirectKeys;
  a.spans = !small && num_splits == 0 && batch <= mla::kPrefillDirectBatch &&
            blocks * num_heads < mla::kPrefillFixedItems * a.pairs &&
            blocks * num_heads * (2 * (int64_t)total_kv / mla::kPrefillTile + 8) < mla::kPrefillDirectUnits;
  a.direct = batch <= mla::kPrefillDirectBatch && (small || a.spans);
  cudaError_t e = a.direct ? cudaSuccess : mla::launch_prefill_plan(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "prefill plan launch");
  e = mla::launch_prefill(tm_q, tm_kv, tm_pe, a, s);
  if (e != cudaSuccess) return cuda_fail(e, "prefill launch");
  if (!a.direct || a.spans) e = mla::launch_prefill_combine(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "prefill combine launch");
  return ok();
}

int mla_prefill_status(const void* workspace, int* status, void* stream) {
  if (!workspace || !status) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  mla::PrefillHeader h;
  cudaError_t e = cudaMemcpyAsync(&h, workspace, sizeof h, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  int bits = h.status;
  for (int i = 0; i < h.ctas && i < 2 * mla::kPrefillMaxPairs; ++i)
    if (h.gave_up[i]) bits |= MLA_DEVERR_TIMEOUT;
  *status = bits;
  return ok();
}

size_t mla_decode_shared_workspace_size(int batch, int prefixes, int total_q, int num_heads, int max_splits) {
  if (batch <= 0 || prefixes <= 0 || total_q <= 0 || num_heads <= 0 || max_splits < 0) return 0;
  return mla::workspace_layout(batch, total_q, num_heads, max_splits, prefixes).total;
}

int mla_decode_shared(const void* q_abs, const void* q_pe, const void* cache, int64_t num_blocks, int page_size,
                      int cache_dtype, float kv_scale, const int32_t* prefix_table, int max_prefix_pages,
                      const int32_t* prefix_lens, const int32_t* prefix_requests, int prefixes,
                      const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens, int batch,
                      const int32_t* query_start_loc, int total_q, int num_heads, float scale, int num_splits,
                      void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || total_q < 0 || prefixes < 0)
    return fail(MLA_ERR_INVALID_ARG, "batch, prefixes and total_q must be >= 0");
  if (num_heads < 1 || num_heads > 1024) return fail(MLA_ERR_INVALID_ARG, "num_heads must be in [1, 1024]");
  if (batch == 0 || total_q == 0) return ok();
  if (prefixes < 1) return fail(MLA_ERR_INVALID_ARG, "a batch needs at least one prefix (its length may be 0)");
  if (batch > kMaxBatch || prefixes > kMaxBatch)
    return fail(MLA_ERR_UNSUPPORTED, "batch and prefixes must be <= %d", kMaxBatch);
  if (!prefix_table || !prefix_lens || !prefix_requests) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(prefix_table, 4) || !aligned(prefix_lens, 4) || !aligned(prefix_requests, 4))
    return fail(MLA_ERR_INVALID_ARG, "prefix_table, prefix_lens and prefix_requests must be 4-byte aligned");
  if (!valid_page_size(page_size))
    return fail(MLA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256 (got %d)", page_size);
  if (max_prefix_pages <= 0) return fail(MLA_ERR_INVALID_ARG, "max_prefix_pages must be positive");
  if (max_pages_per_seq <= 0) return fail(MLA_ERR_INVALID_ARG, "max_pages_per_seq must be positive");
  if ((int64_t)max_prefix_pages * page_size + total_q > kMaxKeys ||
      (int64_t)max_pages_per_seq * page_size + total_q > kMaxKeys)
    return fail(MLA_ERR_UNSUPPORTED, "pages of a table * page_size + total_q must be <= 2^30");
  if (!std::isfinite(scale * 1.4426950408889634f) || scale == 0.f)
    return fail(MLA_ERR_INVALID_ARG, "scale must be nonzero and scale * log2(e) finite");
  if (cache_dtype == MLA_FP8_E4M3 && !std::isnormal(scale * 1.4426950408889634f * kv_scale))
    return fail(MLA_ERR_INVALID_ARG, "scale * kv_scale must be a normal float (the scores' factor)");
  if (num_splits < 0 || num_splits > 4096) return fail(MLA_ERR_INVALID_ARG, "num_splits must be in [0, 4096]");
  const int64_t rows = (int64_t)total_q * num_heads;
  if (rows >= ((int64_t)1 << 30))
    return fail(MLA_ERR_UNSUPPORTED, "total_q * num_heads must be below 2^30");
  if (2 * (rows / mla::kRows + batch + 2) * (num_splits > 1 ? num_splits : 1) * mla::kRows >= (int64_t)1 << 31)
    return fail(MLA_ERR_UNSUPPORTED, "total_q * num_heads * num_splits is too large");
  // the plan's axis: every group of 128 rows with the tiles of its longest keys
  const int64_t tiles = (rows / mla::kRows + batch + 1) * ((int64_t)max_pages_per_seq * page_size / mla::kTile + 8) +
                        (rows / mla::kRows + (prefixes < batch ? prefixes : batch) + 1) *
                            ((int64_t)max_prefix_pages * page_size / mla::kTile + 8);
  if (tiles >= (int64_t)1 << 31)
    return fail(MLA_ERR_UNSUPPORTED, "total_q * num_heads / 128 * the keys of a table / 64 is too large");
  const mla::WorkspaceLayout L = mla::workspace_layout(batch, total_q, num_heads, num_splits, prefixes);
  const int esize = cache_dtype == MLA_FP8_E4M3 ? 1 : 2;
  const Extent outputs[] = {dense(out, rows * mla::kLkv * 2), dense(lse, rows * 4), dense(workspace, (int64_t)L.total)};
  const Extent inputs[] = {dense(q_abs, rows * mla::kLkv * 2),
                           dense(q_pe, rows * mla::kRope * 2),
                           dense(cache, num_blocks * page_size * mla::kDqk * esize),
                           dense(prefix_table, (int64_t)prefixes * max_prefix_pages * 4),
                           dense(prefix_lens, prefixes * 4LL),
                           dense(prefix_requests, (prefixes + 1LL) * 4),
                           dense(block_table, (int64_t)batch * max_pages_per_seq * 4),
                           dense(seq_lens, batch * 4LL),
                           dense(query_start_loc, (batch + 1LL) * 4)};
  if (num_blocks > 0 && num_blocks < (1LL << 31) && any_overlap(outputs, 3, inputs, 9))
    return fail(MLA_ERR_INVALID_ARG, "out, lse and the workspace must not overlap each other or the inputs");
  // A unit's fixed cost in tiles.  A fit of the pairs' times gives 3.5 to 4.6 us a
  // unit, of few rows and of many, and 1.1 a tile; e4m3 rows 5 and 1.6.  Batches of
  // all sizes, over the best of 2 to 7 for each: bf16 1.5 % with 3 and one for each
  // 64 rows (3: 1.9, 4: 2.0, 5: 2.9), e4m3 1.4 with 3 (4: 1.6, 5: 2.6; with one for
  // each 64 rows 2.2)
  const mla::SharedArgs sh{prefix_lens, prefix_requests, prefixes, max_prefix_pages, total_q,
                           tiles,       3,               cache_dtype == MLA_BF16};
  return decode_impl(q_abs, q_pe, nullptr, 0.f, cache, num_blocks, page_size, cache_dtype, kv_scale, block_table,
                     max_pages_per_seq, seq_lens, batch, query_start_loc, total_q, num_heads, scale, num_splits, out,
                     lse, workspace, workspace_bytes, stream, nullptr, nullptr, &sh, prefix_table);
}

int mla_key_weights(const void* q_abs, const void* q_pe, const void* cache, int64_t num_blocks, int page_size,
                    int cache_dtype, float kv_scale, const int32_t* block_table, int max_pages_per_seq,
                    const int32_t* seq_lens, int batch, const int32_t* query_start_loc, int total_q, int num_heads,
                    float scale, const float* lse, float decay, float* weights, int64_t weight_stride, int weight_len,
                    int* status, void* stream) {
  if (batch < 0 || total_q < 0 || weight_len < 0)
    return fail(MLA_ERR_INVALID_ARG, "batch, total_q and weight_len must be >= 0");
  if (num_heads < 1 || num_heads > 1024) return fail(MLA_ERR_INVALID_ARG, "num_heads must be in [1, 1024]");
  if (cache_dtype != MLA_BF16 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_INVALID_ARG, "cache_dtype must be MLA_BF16 or MLA_FP8_E4M3 (got %d)", cache_dtype);
  const bool fp8 = cache_dtype == MLA_FP8_E4M3;
  if (fp8 && !(std::isfinite(kv_scale) && kv_scale > 0.f))
    return fail(MLA_ERR_INVALID_ARG, "kv_scale must be finite and > 0 for an fp8 cache");
  const float factor = scale * 1.4426950408889634f * (fp8 ? kv_scale : 1.f);
  if (!std::isnormal(factor))
    return fail(MLA_ERR_INVALID_ARG, "scale must be nonzero and scale * log2(e) (* kv_scale) a normal float");
  if (!(std::isfinite(decay) && decay >= 0.f)) return fail(MLA_ERR_INVALID_ARG, "decay must be finite and >= 0");
  if (batch == 0 || weight_len == 0) return ok();
  if (!query_start_loc && total_q != batch)
    return fail(MLA_ERR_INVALID_ARG, "without query_start_loc every request has one query token (total_q == batch)");
  if (batch > kMaxBatch) return fail(MLA_ERR_UNSUPPORTED, "batch must be <= %d", kMaxBatch);
  if (!valid_page_size(page_size))
    return fail(MLA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256 (got %d)", page_size);
  if (num_blocks <= 0 || num_blocks * (int64_t)page_size >= (int64_t)1 << 31)
    return fail(MLA_ERR_INVALID_ARG, "num_blocks * page_size must be in [1, 2^31)");
  if (max_pages_per_seq <= 0) return fail(MLA_ERR_INVALID_ARG, "max_pages_per_seq must be positive");
  if ((int64_t)max_pages_per_seq * page_size > kMaxKeys || weight_len > kMaxKeys)
    return fail(MLA_ERR_UNSUPPORTED, "max_pages_per_seq * page_size and weight_len must be <= 2^30");
  const int64_t rows = (int64_t)total_q * num_heads;
  if (rows >= (int64_t)1 << 30) return fail(MLA_ERR_UNSUPPORTED, "total_q * num_heads must be below 2^30");
  if (!cache || !block_table || !seq_lens || !weights || (total_q > 0 && (!q_abs || !q_pe || !lse)))
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(q_abs, 16) || !aligned(q_pe, 16) || !aligned(cache, 16))
    return fail(MLA_ERR_INVALID_ARG, "q_abs, q_pe and cache must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(query_start_loc, 4) || !aligned(lse, 4) ||
      !aligned(weights, 4) || !aligned(status, 4))
    return fail(MLA_ERR_INVALID_ARG, "block_table, seq_lens, query_start_loc, lse, weights and status must be 4-byte aligned");
  if (weight_stride < weight_len || weight_stride > kMaxStride)
    return fail(MLA_ERR_INVALID_ARG, "weight_stride must be in [weight_len, 2^32]");
  const Extent outputs[] = {weight_extent(weights, batch, weight_stride, weight_len), dense(status, 4)};
  const Extent inputs[] = {dense(total_q ? q_abs : nullptr, rows * mla::kLkv * 2),
                           dense(total_q ? q_pe : nullptr, rows * mla::kRope * 2),
                           dense(cache, num_blocks * page_size * mla::kDqk * (fp8 ? 1 : 2)),
                           dense(block_table, (int64_t)batch * max_pages_per_seq * 4),
                           dense(seq_lens, batch * 4LL),
                           dense(query_start_loc, (batch + 1LL) * 4),
                           dense(total_q ? lse : nullptr, rows * 4)};
  if (any_overlap(outputs, 2, inputs, 7))
    return fail(MLA_ERR_INVALID_ARG, "weights and status must not overlap each other or the inputs");
  const int sms = sm_count();
  if (sms < 2) return fail(MLA_ERR_CUDA, "cannot query the current device");
  // Columns of a product: a request's query rows (of an average one, where
  // query_start_loc says) in as few tiles of at most 256 as hold them, a
  // multiple of 32; each CTA of a pair loads half of them
  const int64_t per_request = (total_q + (int64_t)batch - 1) / batch * num_heads;
  const int64_t row_tiles = per_request > 256 ? (per_request + 255) / 256 : 1;
  int row_tile = (int)((per_request + row_tiles - 1) / row_tiles + 31) / 32 * 32;
  if (row_tile < 32) row_tile = 32;
  CUtensorMap tm_q, tm_qr, tm_kv;
  bool enc = mla::encode_tmap_2d(&tm_kv, cache, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                 mla::kDqk, (uint64_t)num_blocks * page_size, mla::kDqk * (fp8 ? 1 : 2), fp8 ? 192 : 64,
                                 page_size < (fp8 ? 32 : 128) ? page_size : (fp8 ? 32 : 128),
                                 fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
  tm_q = tm_qr = tm_kv;   // without a query row none is loaded
  if (total_q > 0)
    enc = enc &&
          mla::encode_tmap_2d(&tm_q, q_abs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kLkv, rows, mla::kLkv * 2, 64,
                              row_tile / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
          mla::encode_tmap_2d(&tm_qr, q_pe, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, mla::kRope, rows, mla::kRope * 2, 64,
                              row_tile / 2, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!enc) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor layout");
  mla::KeyWeightArgs a{};
  a.cache = static_cast<const uint8_t*>(cache);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.qsl = query_start_loc;
  a.lse = lse;
  a.weights = weights;
  a.weight_stride = weight_stride;
  a.weight_len = weight_len;
  a.batch = batch;
  a.total_q = total_q;
  a.num_heads = num_heads;
  a.max_pages = max_pages_per_seq;
  a.page_size = page_size;
  a.num_blocks = num_blocks;
  a.scale_log2 = factor;
  a.decay = decay;
  a.row_tile = row_tile;
  a.many_rows = row_tiles > 1;
  a.status = status;
  a.wait_limit_ns = g_wait_limit_ns;
  a.debug_skip_tile = g_test_skip_tile;
  cudaError_t e = mla::launch_key_weights(tm_q, tm_qr, tm_kv, fp8, a, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "key weights launch");
  return ok();
}

int mla_evict_select(const float* weights, int64_t weight_stride, int weight_len, const int32_t* seq_lens, int batch,
                     int budget, int sinks, int recent, int32_t* keep, int32_t* keep_lens, int* status, void* stream) {
  if (batch < 0 || weight_len < 0) return fail(MLA_ERR_INVALID_ARG, "batch and weight_len must be >= 0");
  if (budget < 1) return fail(MLA_ERR_INVALID_ARG, "budget must be positive (got %d)", budget);
  if (sinks < 0 || recent < 0 || sinks > budget || recent > budget - sinks)
    return fail(MLA_ERR_INVALID_ARG, "sinks and recent must be >= 0 and sinks + recent <= budget");
  if (batch == 0) return ok();
  if (batch > kMaxBatch) return fail(MLA_ERR_UNSUPPORTED, "batch must be <= %d", kMaxBatch);
  if (weight_len > kMaxKeys || budget > kMaxKeys)
    return fail(MLA_ERR_UNSUPPORTED, "weight_len and budget must be <= 2^30");
  if ((weight_len > 0 && !weights) || !seq_lens || !keep || !keep_lens)
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(weights, 4) || !aligned(seq_lens, 4) || !aligned(keep, 4) || !aligned(keep_lens, 4) ||
      !aligned(status, 4))
    return fail(MLA_ERR_INVALID_ARG, "tensors must be 4-byte aligned");
  if (weight_stride < weight_len || weight_stride > kMaxStride)
    return fail(MLA_ERR_INVALID_ARG, "weight_stride must be in [weight_len, 2^32]");
  const bool in_place = keep_lens == seq_lens;
  const Extent outputs[] = {dense(keep, (int64_t)batch * budget * 4), dense(keep_lens, batch * 4LL), dense(status, 4)};
  const Extent inputs[] = {weight_extent(weights, batch, weight_stride, weight_len),
                           dense(in_place ? nullptr : seq_lens, batch * 4LL)};
  if (any_overlap(outputs, 3, inputs, 2))
    return fail(MLA_ERR_INVALID_ARG,
                "keep, keep_lens and status must not overlap each other or the inputs (keep_lens may be seq_lens itself)");
  const int sms = sm_count();
  if (sms < 1) return fail(MLA_ERR_CUDA, "cannot query the current device");
  const mla::SelectArgs a{weights, weight_stride, weight_len, seq_lens, batch, budget,
                          sinks,   recent,        keep,       keep_lens, status};
  cudaError_t e = mla::launch_select(a, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "selection launch");
  return ok();
}

int mla_cache_compact(void* cache, int64_t num_blocks, int page_size, int cache_dtype, const int32_t* block_table,
                      int max_pages_per_seq, const int32_t* keep, int max_keep, const int32_t* keep_lens, int batch,
                      float* weights, int64_t weight_stride, int weight_len, int* status, void* stream) {
  if (batch < 0 || max_keep < 0) return fail(MLA_ERR_INVALID_ARG, "batch and max_keep must be >= 0");
  if (cache_dtype != MLA_BF16 && cache_dtype != MLA_FP8_E4M3)
    return fail(MLA_ERR_INVALID_ARG, "cache_dtype must be MLA_BF16 or MLA_FP8_E4M3 (got %d)", cache_dtype);
  if (page_size <= 0 || num_blocks <= 0 || max_pages_per_seq <= 0 || num_blocks > ((1LL << 31) - 1) / page_size)
    return fail(MLA_ERR_INVALID_ARG,
                "page_size, num_blocks and max_pages_per_seq must be positive and num_blocks * page_size < 2^31");
  if (batch == 0 || max_keep == 0) return ok();
  if (batch > kMaxBatch) return fail(MLA_ERR_UNSUPPORTED, "batch must be <= %d", kMaxBatch);
  if (max_keep > kMaxKeys) return fail(MLA_ERR_UNSUPPORTED, "max_keep must be <= 2^30");
  if (!cache || !block_table || !keep || !keep_lens) return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned(cache, 16)) return fail(MLA_ERR_INVALID_ARG, "cache must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(keep, 4) || !aligned(keep_lens, 4) || !aligned(weights, 4) ||
      !aligned(status, 4))
    return fail(MLA_ERR_INVALID_ARG, "block_table, keep, keep_lens, weights and status must be 4-byte aligned");
  if (weights && (weight_len < 1 || weight_len > kMaxKeys || weight_stride < weight_len || weight_stride > kMaxStride))
    return fail(MLA_ERR_INVALID_ARG, "weight_len must be in [1, 2^30] and weight_stride in [weight_len, 2^32]");
  const int row_bytes = mla::kDqk * (cache_dtype == MLA_FP8_E4M3 ? 1 : 2);
  const Extent outputs[] = {dense(cache, num_blocks * page_size * row_bytes),
                            weight_extent(weights, batch, weight_stride, weight_len), dense(status, 4)};
  const Extent inputs[] = {dense(block_table, (int64_t)batch * max_pages_per_seq * 4),
                           dense(keep, (int64_t)batch * max_keep * 4), dense(keep_lens, batch * 4LL)};
  if (any_overlap(outputs, 3, inputs, 3))
    return fail(MLA_ERR_INVALID_ARG, "cache, weights and status must not overlap each other or the inputs");
  const int sms = sm_count();
  if (sms < 1) return fail(MLA_ERR_CUDA, "cannot query the current device");
  const mla::CompactArgs a{static_cast<uint8_t*>(cache), num_blocks, page_size, block_table, max_pages_per_seq, keep,
                           keep_lens, batch, max_keep, weights, weight_stride, weight_len, status,
                           g_wait_limit_ns, g_test_skip_tile};
  cudaError_t e = mla::launch_compact(a, row_bytes, sms, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_fail(e, "compaction launch");
  return ok();
}

}  // extern "C"
