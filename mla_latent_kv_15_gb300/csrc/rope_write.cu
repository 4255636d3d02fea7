// Append of the step's latent rows to the paged cache with the position
// rotation on the way (mla_rope_cache_write).  Per token, with the table row
// (cos, sin) of its position:
//
//   c     = kv_c                                   (no norm weight)
//         = kv_c * g / sqrt(mean(kv_c^2) + eps)    (with one)
//   row   = [c | rot(k_pe)]  -> cache slot (bf16 or e4m3(row / kv_scale)), latent row (bf16)
//   q_out = rot(q_pe) of every head
//   rot:    (x_i, x_j) -> (x_i cos_k - x_j sin_k, x_j cos_k + x_i sin_k)
//           over the pairs (i, j) = (2k, 2k+1) or (k, k+32), k < 32
//
// Everything is computed in float32 from the bf16 inputs and rounded once, to
// the type it is stored in.  The op moves bytes (a token of 128 heads reads and
// writes 16 KB of query and 1.1 KB of latent row each way), so it is bound by
// HBM for prompts and by latency for a decode step.  One warp takes one
// token's latent row, or 32 heads of one token's query: a thread holds two
// 16-byte vectors of a 64-dim rope row, dims 8v.. and 8v+32.., which hold both
// partners of its pairs in either pairing, and has four heads' loads in flight
// (8192 tokens of 128 heads with latent rows, about 8 us of graph launch
// included: 8 heads a warp 68.7 us, 16: 60.5, 32: 52.4, 64: 56.5; 299 MB at the
// copy rate are 44).  The data is loaded before the position is known, so the
// two latencies overlap.  (A call among others: 44.7 us, 99 % of the copy rate;
// 64 tokens 3.3 us in a graph.)
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_rows.cuh"
#include "common.cuh"

namespace mla {
namespace {

__device__ __forceinline__ void unpack8(const uint4 v, float (&x)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __bfloat1622float2(h[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint4 v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return v;
}

// Plain loads throughout: the kernel may start beside the one before it (a
// programmatic dependent), which may still be writing what this one reads, and
// the read-only path is for memory that nobody writes while the kernel runs.

// The table entries a thread's two vectors (dims 8v.. and 8v+32.., v < 4) need.
// Pairs (2k, 2k+1): entries 4v..4v+3 for the first vector, 4v+16.. for the
// second; pairs (k, k+32): entries 8v..8v+7 for both.
struct Turn {
  float cos[8], sin[8];
};

template <bool kPairs>
__device__ __forceinline__ Turn load_turn(const float* row, int v) {
  Turn t;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = kPairs ? 4 * v + 16 * h : 8 * v + 4 * h;
    const float4 c = *reinterpret_cast<const float4*>(row + at);
    const float4 s = *reinterpret_cast<const float4*>(row + 32 + at);
    t.cos[4 * h] = c.x, t.cos[4 * h + 1] = c.y, t.cos[4 * h + 2] = c.z, t.cos[4 * h + 3] = c.w;
    t.sin[4 * h] = s.x, t.sin[4 * h + 1] = s.y, t.sin[4 * h + 2] = s.z, t.sin[4 * h + 3] = s.w;
  }
  return t;
}

// Rotate the two vectors a (dims 8v..) and b (dims 8v+32..) in place.
template <bool kPairs>
__device__ __forceinline__ void turn_by(float (&a)[8], float (&b)[8], const Turn& t) {
  if (kPairs) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = a[2 * k], y = a[2 * k + 1];
      a[2 * k] = x * t.cos[k] - y * t.sin[k];
      a[2 * k + 1] = y * t.cos[k] + x * t.sin[k];
      const float z = b[2 * k], w = b[2 * k + 1];
      b[2 * k] = z * t.cos[4 + k] - w * t.sin[4 + k];
      b[2 * k + 1] = w * t.cos[4 + k] + z * t.sin[4 + k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = a[k], y = b[k];
      a[k] = x * t.cos[k] - y * t.sin[k];
      b[k] = y * t.cos[k] + x * t.sin[k];
    }
  }
}

// Eight values of a cache row (vector v of its 72) as the cache's type.
template <bool kFp8>
__device__ __forceinline__ void store_cache8(const RopeWriteArgs& w, int64_t slot, int v, const float (&x)[8]) {
  if (kFp8) {
    float lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      lo[k] = __fdiv_rn(x[k], w.kv_scale);
      hi[k] = __fdiv_rn(x[4 + k], w.kv_scale);
    }
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(w.cache) + slot * kDqk)[v] = make_uint2(fp8x4(lo), fp8x4(hi));
  } else {
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(w.cache) + slot * kDqk)[v] = pack8(x);
  }
}

// One warp: token `tok`'s latent row.
template <bool kFp8, bool kPairs>
__device__ __forceinline__ void latent_row(const RopeWriteArgs& w, int64_t tok, int lane) {
  const int64_t pos = w.positions[tok];
  const int64_t slot = w.slots[tok];
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w.kv_c) + tok * w.kv_c_stride);
  const uint4* pe = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w.k_pe) + tok * w.k_pe_stride);
  const uint4 v0 = src[lane], v1 = src[lane + 32];
  uint4 pa, pb;
  if (lane < 4) pa = pe[lane], pb = pe[lane + 4];
  const bool bad = pos < 0 || pos >= w.max_positions;
  if (bad) {
    if (lane == 0 && w.status) atomicOr(w.status, 16);   // MLA_DEVERR_BAD_POSITION
    return;
  }
  const bool keep = slot >= 0 && slot < w.num_slots;
  float x0[8], x1[8];
  float a[8], b[8];
  if (lane < 4) {
    unpack8(pa, a);
    unpack8(pb, b);
    turn_by<kPairs>(a, b, load_turn<kPairs>(w.cos_sin + pos * kRope, lane));
  }
  unpack8(v0, x0);
  unpack8(v1, x1);
  if (w.norm_weight) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += x0[k] * x0[k] + x1[k] * x1[k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = 1.0f / sqrtf(ss * (1.0f / kLkv) + w.norm_eps);
    const uint4* g = static_cast<const uint4*>(w.norm_weight);
    float g0[8], g1[8];
    unpack8(g[lane], g0);
    unpack8(g[lane + 32], g1);
#pragma unroll
    for (int k = 0; k < 8; ++k) x0[k] = x0[k] * r * g0[k], x1[k] = x1[k] * r * g1[k];
  }
  // every lane holds its inputs by now: the latent row may be the input row
  __syncwarp();
  if (keep) {
    store_cache8<kFp8>(w, slot, lane, x0);
    store_cache8<kFp8>(w, slot, lane + 32, x1);
    if (lane < 4) {
      store_cache8<kFp8>(w, slot, 64 + lane, a);
      store_cache8<kFp8>(w, slot, 68 + lane, b);
    }
  }
  if (w.latent) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(w.latent) + tok * w.latent_stride);
    dst[lane] = pack8(x0);
    dst[lane + 32] = pack8(x1);
    if (lane < 4) {
      dst[64 + lane] = pack8(a);
      dst[68 + lane] = pack8(b);
    }
  }
}

// One warp: kWarpHeads heads of token `tok`, four threads per head.
constexpr int kIters = 4, kWarpHeads = 8 * kIters;

template <bool kPairs>
__device__ __forceinline__ void query_rows(const RopeWriteArgs& w, int64_t tok, int group, int lane) {
  const int64_t pos = w.positions[tok];
  const int v = lane & 3, h0 = group * kWarpHeads + (lane >> 2);
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(w.q_pe) + tok * w.q_token_stride;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(w.q_out) + tok * w.qo_token_stride;
  uint4 va[kIters], vb[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int h = h0 + 8 * i;
    if (h < w.num_heads) {
      const uint4* p = reinterpret_cast<const uint4*>(src + h * w.q_head_stride);
      va[i] = p[v];
      vb[i] = p[v + 4];
    }
  }
  if (pos < 0 || pos >= w.max_positions) return;         // flagged by the token's latent row
  const Turn t = load_turn<kPairs>(w.cos_sin + pos * kRope, v);
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int h = h0 + 8 * i;
    if (h < w.num_heads) {
      float a[8], b[8];
      unpack8(va[i], a);
      unpack8(vb[i], b);
      turn_by<kPairs>(a, b, t);
      uint4* p = reinterpret_cast<uint4*>(dst + h * w.qo_head_stride);
      p[v] = pack8(a);
      p[v + 4] = pack8(b);
    }
  }
}

// Warp u of the grid: token u / per, part u % per (0: the latent row, 1..: query heads).
template <bool kFp8, bool kPairs>
__global__ void __launch_bounds__(256) rope_write_kernel(const RopeWriteArgs w, int per) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t u = blockIdx.x * 8LL + (threadIdx.x >> 5);
  const int64_t tok = u / per;
  if (tok >= w.num_tokens) return;
  const int part = (int)(u - tok * per), lane = threadIdx.x & 31;
  if (part == 0)
    latent_row<kFp8, kPairs>(w, tok, lane);
  else
    query_rows<kPairs>(w, tok, part - 1, lane);
}

template <bool kFp8, bool kPairs>
cudaError_t launch_one(const RopeWriteArgs& w, cudaStream_t s) {
  const int per = 1 + (w.q_pe ? (w.num_heads + kWarpHeads - 1) / kWarpHeads : 0);
  const int64_t blocks = (w.num_tokens * per + 7) / 8;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, rope_write_kernel<kFp8, kPairs>, w, per);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_write(const RopeWriteArgs& w, int fp8, int pairs, cudaStream_t s) {
  if (fp8) return pairs ? launch_one<true, true>(w, s) : launch_one<true, false>(w, s);
  return pairs ? launch_one<false, true>(w, s) : launch_one<false, false>(w, s);
}

}  // namespace mla
