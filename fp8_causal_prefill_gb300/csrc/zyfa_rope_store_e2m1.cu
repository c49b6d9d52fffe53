// Rotary positions fused with the store into a 4-bit paged cache: e2m1 codes and one e4m3 scale for each 16 channels.
//
// For 16 neighbouring channels z of a token and head, over the descale: scale = e4m3(max|z| / 6), so that the largest magnitude
// meets the largest code, and code = e2m1(z / scale).  The reciprocals of the descale and of the scale are rounded once and multiplied
// by, as in the e4m3 store, so a value within 2^-22 of the middle between two codes may take either.
//
// Angles, tables and the walk over a block's tokens are those of the e4m3 and bf16 store (rope.cuh).  A thread keeps 8 channels and
// their partners half the rotated width away (or 16 neighbours, where pairs are neighbours), of queries and then of keys.  A block of 16
// keys' channels is then in one thread, or its halves are in two lanes, which tell one another their largest magnitude: nothing is read
// twice.  Where a rotated part begins or ends inside such a block a thread has a block of a key and reads its partners again, by the line
// that its neighbour also reads.  32768 tokens of 32 query and 8 KV heads of 128 channels, dense rows written as well: 129 us, 96% of what
// their bytes take; 173 us by second reads.  Few query heads leave the arithmetic of blocks and angles in sight: 20000 tokens of 8 and 8
// heads take 38 us where their bytes take 28.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "paged.cuh"
#include "rope.cuh"

namespace {

using namespace zyfa::rope;

// Blocks an SM is to hold of 256 (192 for 192 channels) threads where keys go the way of queries: 64 registers, below which they spill
constexpr int kBlocks = 4, kBlocksOf192 = 5;

struct Store4Args {
  const __nv_bfloat16 *q, *k, *v;
  long long q_tok, k_tok, v_tok;  // elements
  __nv_bfloat16 *q_out, *k_out, *v_out;
  const int* positions;
  long long pos_stride;
  const long long* slots;
  const float* inv_freq;
  const float *k_desc, *v_desc;
  int* status;
  long long N;
  zyfa::CacheView cache;
  zyfa::ScaleView scales;
  int H;
  int rot, offset, axis_end[4];
  int desc_per_head;
  int tokens;  // per block
};

__device__ __forceinline__ uint4 bf16x8(const float* y) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest magnitude among 8 values, as bits, whose order is that of magnitudes, with NaN above all.
__device__ __forceinline__ uint32_t top_of(const float* z) {
  float top;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(z[0]), "f"(z[1]), "f"(z[2]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(z[3]), "f"(z[4]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(z[5]), "f"(z[6]));
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(top) : "f"(top), "f"(z[7]), "f"(z[7]));
  return __float_as_uint(top);
}
// What values are multiplied by under a scale; 0 under 0 and NaN.
__device__ __forceinline__ float reciprocal(uint32_t s8) {
  float s;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(s) : "r"(zyfa::widen_e4m3(s8)));
  return s > 0.0f ? __frcp_rn(s) : 0.0f;
}
// The scale of a block with this largest magnitude; *r: what its values are multiplied by, of those in shared memory for each scale.
__device__ __forceinline__ uint8_t scale_of(uint32_t top, const float* reciprocals, float* r) {
  uint16_t s8;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.0f), "f"(__uint_as_float(top) * (1.0f / 6.0f)));
  *r = reciprocals[s8 & 0x7f];
  return static_cast<uint8_t>(s8);
}
__device__ __forceinline__ void times8(float* z, float f) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 p = zyfa::times(z[i], z[i + 1], f);
    z[i] = p.x;
    z[i + 1] = p.y;
  }
}
// Eight e2m1 codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t codes8(const float* z, float r) {
  uint32_t d;
  const float2 x = zyfa::times(z[0], z[1], r), y = zyfa::times(z[2], z[3], r), u = zyfa::times(z[4], z[5], r), v = zyfa::times(z[6], z[7], r);
  asm("{\n\t.reg .b8 a, b, c, e;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\tmov.b32 %0, {a, b, c, e};\n\t}"
      : "=r"(d)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(u.x), "f"(u.y), "f"(v.x), "f"(v.y));
  return d;
}
// 16 values as codes and their scale.
__device__ __forceinline__ void quantise(float (&y)[16], float inv, const float* reciprocals, uint2* codes, uint8_t* scale) {
  times8(y, inv);
  times8(y + 8, inv);
  float r;
  *scale = scale_of(max(top_of(y), top_of(y + 8)), reciprocals, &r);
  *codes = make_uint2(codes8(y, r), codes8(y + 8, r));
}

// NEAT: no block of 16 key channels is rotated in part, or lies in both halves of the rotated part: keys go the way of queries.  Else a
// thread has a block of a key and reads its partners a second time.
template <bool INTERLEAVED, bool NEAT, int DQK, int DV>
__global__ void __launch_bounds__(kThreads<DQK>, NEAT ? (DQK == 192 ? kBlocksOf192 : kBlocks) : 1) store4_kernel(const __grid_constant__ Store4Args a) {
  constexpr int kN = kThreads<DQK>, kPieces = DQK / 16, kBlocksK = DQK / 16, kBlocksV = DV / 16, kHalf = DQK / 2;
  static_assert(kN % kPieces == 0 && kN % kBlocksV == 0);
  __shared__ __align__(16) float s_cos[kMaxTokens][kHalf], s_sin[kMaxTokens][kHalf];
  __shared__ long long s_page[kMaxTokens];  // -1: outside the cache, -2: padding
  __shared__ int s_off[kMaxTokens];
  __shared__ float s_reciprocal[128];
  const int tid = threadIdx.x;
  const long long n0 = static_cast<long long>(blockIdx.x) * a.tokens;
  const int here = static_cast<int>(min(static_cast<long long>(a.tokens), a.N - n0));
  const int H_kv = a.cache.H_kv, half = a.rot / 2;

  // queries: this thread's 8 channels and their partners, or 16 neighbours, the same of every head
  const int j = tid % kPieces;
  int pair = -1, d0, d1;
  if (j * 8 < half) {
    pair = j * 8;
    d0 = a.offset + (INTERLEAVED ? j * 16 : j * 8);
    d1 = INTERLEAVED ? d0 + 8 : d0 + half;
  } else {  // the plain channels in order, eight by eight
    const int d = 16 * j - a.rot;
    d0 = d < a.offset ? d : d + a.rot;
    d1 = d + 8 < a.offset ? d + 8 : d + 8 + a.rot;
  }
  const int heads_q = a.q ? a.H : 0;
  Walk w = {0, tid / kPieces, heads_q + (NEAT && a.k ? H_kv : 0), kN / kPieces};
  if (w.heads) w.settle(); else w.token = here;
  uint4 x0, x1;
  auto fetch = [&]() {
    if (w.token >= here) return;
    const long long n = n0 + w.token;
    const __nv_bfloat16* x = w.head < heads_q ? a.q + n * a.q_tok + w.head * DQK : a.k + n * a.k_tok + (w.head - heads_q) * DQK;
    x0 = *reinterpret_cast<const uint4*>(x + d0);
    x1 = *reinterpret_cast<const uint4*>(x + d1);
  };
  // keys (not NEAT): this thread's block of 16 channels, two halves of 8 that turn alike; from: the channel of a half's partners (its own: none)
  const int kd = tid % kBlocksK * 16;
  int from[2], first_pair[2];
  bool second[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int d = kd + 8 * i, r = d - a.offset;
    const bool turns = r >= 0 && r < a.rot;
    second[i] = turns && !INTERLEAVED && r >= half;
    from[i] = !turns || INTERLEAVED ? d : second[i] ? d - half : d + half;
    first_pair[i] = !turns ? -1 : INTERLEAVED ? r / 2 : second[i] ? r - half : r;
  }
  Walk wk = {0, tid / kBlocksK, H_kv, kN / kBlocksK};
  wk.settle();
  uint4 k0, k1, p0, p1;
  auto fetch_k = [&]() {
    if (wk.token >= here) return;
    const __nv_bfloat16* x = a.k + (n0 + wk.token) * a.k_tok + wk.head * DQK;
    k0 = *reinterpret_cast<const uint4*>(x + kd);
    k1 = *reinterpret_cast<const uint4*>(x + kd + 8);
    if (!INTERLEAVED) {
      p0 = *reinterpret_cast<const uint4*>(x + from[0]);
      p1 = *reinterpret_cast<const uint4*>(x + from[1]);
    }
  };
  const int vd = tid % kBlocksV * 16;
  Walk wv = {0, tid / kBlocksV, H_kv, kN / kBlocksV};
  wv.settle();
  if (!a.k) wv.token = here;
  if (!a.k || NEAT) wk.token = here;
  uint4 v0, v1;
  auto fetch_v = [&]() {
    if (wv.token >= here) return;
    const __nv_bfloat16* x = a.v + (n0 + wv.token) * a.v_tok + wv.head * DV + vd;
    v0 = *reinterpret_cast<const uint4*>(x);
    v1 = *reinterpret_cast<const uint4*>(x + 8);
  };
  zyfa::wait_for_predecessor();
  // the first loads run while the tables are made
  fetch();
  if (!NEAT) fetch_k();
  fetch_v();
  if (tid < here) {
    const long long slot = a.slots[n0 + tid];
    long long at = -2, off = 0;
    if (slot >= 0) {
      place_of(slot, a.cache.page_size, &at, &off);
      if (at >= a.cache.num_pages) {
        at = -1;
        if (a.k) atomicOr(a.status, zyfa::kStatusBadPageBit);
      }
    }
    s_page[tid] = at;
    s_off[tid] = static_cast<int>(off);
  }
  if (tid < 128 && a.k) s_reciprocal[tid] = reciprocal(tid);
  fill_turns<kN>(a, n0, here, s_cos, s_sin);
  const float inv_k = a.desc_per_head ? 0.0f : inverse(a.k_desc, 0), inv_v = a.desc_per_head ? 0.0f : inverse(a.v_desc, 0);
  __syncthreads();

  while (wv.token < here) {
    const int token = wv.token, head = wv.head;
    const uint4 c0 = v0, c1 = v1;
    wv.head += wv.lanes;
    wv.settle();
    fetch_v();
    const long long at = s_page[token];
    if (at == -2) continue;
    if (a.v_out) {
      uint4* to = reinterpret_cast<uint4*>(a.v_out + ((n0 + token) * H_kv + head) * DV + vd);
      to[0] = c0;
      to[1] = c1;
    }
    if (at < 0) continue;
    float y[16];
    widen8(c0, *reinterpret_cast<float(*)[8]>(y));
    widen8(c1, *reinterpret_cast<float(*)[8]>(y + 8));
    uint2 codes;
    uint8_t scale;
    quantise(y, a.desc_per_head ? inverse(a.v_desc, head) : inv_v, s_reciprocal, &codes, &scale);
    *reinterpret_cast<uint2*>(a.cache.v + at * a.cache.v_page + s_off[token] * a.cache.v_tok + head * a.cache.v_head + vd / 2) = codes;
    a.scales.v[at * a.scales.v_page + s_off[token] * a.scales.v_tok + head * a.scales.v_head + vd / 16] = scale;
  }
  while (!NEAT && wk.token < here) {
    const int token = wk.token, head = wk.head;
    float y[16], p[16];
    widen8(k0, *reinterpret_cast<float(*)[8]>(y));
    widen8(k1, *reinterpret_cast<float(*)[8]>(y + 8));
    if (!INTERLEAVED) {
      widen8(p0, *reinterpret_cast<float(*)[8]>(p));
      widen8(p1, *reinterpret_cast<float(*)[8]>(p + 8));
    }
    wk.head += wk.lanes;
    wk.settle();
    fetch_k();
    const long long at = s_page[token];
    if (at == -2) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (first_pair[i] < 0) continue;
      float* z = y + 8 * i;
      const float *c = &s_cos[token][first_pair[i]], *s = &s_sin[token][first_pair[i]];
      if (INTERLEAVED) {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float u = z[2 * m], v = z[2 * m + 1];
          z[2 * m] = fmaf(u, c[m], v * -s[m]);
          z[2 * m + 1] = fmaf(u, s[m], v * c[m]);
        }
      } else {
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float u = z[m], v = p[8 * i + m];
          z[m] = second[i] ? fmaf(v, s[m], u * c[m]) : fmaf(u, c[m], v * -s[m]);
        }
      }
    }
    if (a.k_out) {
      uint4* to = reinterpret_cast<uint4*>(a.k_out + ((n0 + token) * H_kv + head) * DQK + kd);
      to[0] = bf16x8(y);
      to[1] = bf16x8(y + 8);
    }
    if (at < 0) continue;
    uint2 codes;
    uint8_t scale;
    quantise(y, a.desc_per_head ? inverse(a.k_desc, head) : inv_k, s_reciprocal, &codes, &scale);
    *reinterpret_cast<uint2*>(a.cache.k + at * a.cache.k_page + s_off[token] * a.cache.k_tok + head * a.cache.k_head + kd / 2) = codes;
    a.scales.k[at * a.scales.k_page + s_off[token] * a.scales.k_tok + head * a.scales.k_head + kd / 16] = scale;
  }
  while (w.token < here) {
    const int token = w.token, head = w.head;
    float u[8], v[8];
    widen8(x0, u);
    widen8(x1, v);
    w.head += w.lanes;
    w.settle();
    fetch();
    const long long at = s_page[token];
    if (at == -2) continue;
    if (pair >= 0) {
      float c[8], s[8];
      *reinterpret_cast<float4*>(c) = *reinterpret_cast<const float4*>(&s_cos[token][pair]);
      *reinterpret_cast<float4*>(c + 4) = *reinterpret_cast<const float4*>(&s_cos[token][pair + 4]);
      *reinterpret_cast<float4*>(s) = *reinterpret_cast<const float4*>(&s_sin[token][pair]);
      *reinterpret_cast<float4*>(s + 4) = *reinterpret_cast<const float4*>(&s_sin[token][pair + 4]);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        if constexpr (INTERLEAVED) {  // pairs are neighbours of u, then of v
          float* y = i < 4 ? u + 2 * i : v + 2 * i - 8;
          rotate2(y[0], y[2], y[1], y[3], c + i, s + i);
        } else {
          rotate2(u[i], u[i + 1], v[i], v[i + 1], c + i, s + i);
        }
      }
    }
    const long long n = n0 + token;
    if (!NEAT || head < heads_q) {
      __nv_bfloat16* row = a.q_out + (n * a.H + head) * DQK;
      *reinterpret_cast<uint4*>(row + d0) = bf16x8(u);
      *reinterpret_cast<uint4*>(row + d1) = bf16x8(v);
    } else {
      const int hk = head - heads_q;
      if (a.k_out) {
        __nv_bfloat16* row = a.k_out + (n * H_kv + hk) * DQK;
        *reinterpret_cast<uint4*>(row + d0) = bf16x8(u);
        *reinterpret_cast<uint4*>(row + d1) = bf16x8(v);
      }
      if (at < 0) continue;
      const float inv = a.desc_per_head ? inverse(a.k_desc, hk) : inv_k;
      times8(u, inv);
      times8(v, inv);
      uint32_t tu = top_of(u), tv = top_of(v);
      const bool apart = !INTERLEAVED && pair >= 0;  // u and v are halves of two blocks, whose others the next lane has
      if (apart) {
        const unsigned both = 3u << (tid & 30);
        tu = max(tu, __shfl_xor_sync(both, tu, 1));
        tv = max(tv, __shfl_xor_sync(both, tv, 1));
      } else {
        tu = tv = max(tu, tv);
      }
      float ru, rv;
      const uint8_t su = scale_of(tu, s_reciprocal, &ru), sv = scale_of(tv, s_reciprocal, &rv);
      uint8_t* codes = a.cache.k + at * a.cache.k_page + s_off[token] * a.cache.k_tok + hk * a.cache.k_head;
      uint8_t* scales = a.scales.k + at * a.scales.k_page + s_off[token] * a.scales.k_tok + hk * a.scales.k_head;
      *reinterpret_cast<uint32_t*>(codes + d0 / 2) = codes8(u, ru);
      *reinterpret_cast<uint32_t*>(codes + d1 / 2) = codes8(v, rv);
      if (!apart || !(d0 & 8)) {
        scales[d0 / 16] = su;
        if (apart) scales[d1 / 16] = sv;
      }
    }
  }
}

// Tokens a block: so many that all blocks run at once, in as few such waves as 12 to 32 tokens of a few or more heads allow (8000 tokens of 8
// heads of 192/128: 21.2 us in one wave, 26.1 where an eighth of the blocks waits).  An SM holds 4 blocks (5 of 192 channels) where keys
// go the way of queries, 2 to 4 where a thread has a block of a key: 8000 tokens of 8 heads of 192/128 whose 48 channels from 136 on turn take
// 32.8 us in waves of 3 blocks, 37.2 in waves of 5; 32768 of 32 and 8 heads of 128 with 48 148.0 (2) and 152.7 (4).
template <bool INTERLEAVED, bool NEAT, int DQK, int DV>
cudaError_t launch_of(Store4Args& a, int dev, cudaStream_t stream) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> held[kMaxDevices];
  int blocks = dev < kMaxDevices ? held[dev].load(std::memory_order_relaxed) : 0;
  if (blocks == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, store4_kernel<INTERLEAVED, NEAT, DQK, DV>, kThreads<DQK>, 0);
    if (e != cudaSuccess) return e;
    blocks = std::max(blocks, 1);
    if (dev < kMaxDevices) held[dev].store(blocks, std::memory_order_relaxed);
  }
  const long long at_once = static_cast<long long>(blocks) * std::max(1, zyfa::device_sm_count(dev));
  const long long most = std::min(kMaxTokens, std::max(12, 320 / (a.H + 2 * a.cache.H_kv))), waves = (a.N + most * at_once - 1) / (most * at_once);
  a.tokens = static_cast<int>((a.N + at_once * waves - 1) / (at_once * waves));
  const dim3 grid(static_cast<unsigned>((a.N + a.tokens - 1) / a.tokens));
  return zyfa::launch_dependent(store4_kernel<INTERLEAVED, NEAT, DQK, DV>, grid, kThreads<DQK>, 0, stream, a);
}

template <bool INTERLEAVED, bool NEAT>
cudaError_t launch(Store4Args& a, int D_qk, int dev, cudaStream_t stream) {
  return D_qk == 64    ? launch_of<INTERLEAVED, NEAT, 64, 64>(a, dev, stream)
         : D_qk == 128 ? launch_of<INTERLEAVED, NEAT, 128, 128>(a, dev, stream)
                       : launch_of<INTERLEAVED, NEAT, 192, 128>(a, dev, stream);
}

template <bool INTERLEAVED>
cudaError_t launch(Store4Args& a, bool neat, int D_qk, int dev, cudaStream_t stream) {
  return neat ? launch<INTERLEAVED, true>(a, D_qk, dev, stream) : launch<INTERLEAVED, false>(a, D_qk, dev, stream);
}

}  // namespace

extern "C" zyfa_status_t zyfa_rope_paged_store_e2m1(const void* q, const void* k, const void* v, long long q_token_stride,
                                                    long long k_token_stride, long long v_token_stride, void* q_out, void* k_out,
                                                    void* v_out, const int* positions, long long position_stride,
                                                    const long long* slots, long long N, int H, const zyfa_paged_cache_t* cache,
                                                    const zyfa_paged_scales_t* scales, const zyfa_rope_t* rope, const float* k_descale,
                                                    const float* v_descale, int descale_per_kv_head, cudaStream_t stream) {
  using zyfa::aligned;
  Store4Args a = {};
  zyfa_status_t st = zyfa::check_cache(cache, &a.cache, zyfa::k4BitCaches);
  if (st == ZYFA_OK) st = zyfa::check_scales(scales, &a.scales);
  if (st != ZYFA_OK) return st;
  const int H_kv = cache->H_kv, D_qk = cache->D_qk, D_v = cache->D_v;
  if (N < 0 || H < 1 || H % H_kv != 0 || (descale_per_kv_head != 0 && descale_per_kv_head != 1)) return ZYFA_ERR_INVALID_ARG;
  if (!k != !v || (!q && !k)) return ZYFA_ERR_INVALID_ARG;
  // cache and scales are written here: no row of one of the four may overlap another
  const CacheDims dims[4] = {{*cache, cache->k_page_stride, cache->k_token_stride, cache->k_head_stride},
                             {*cache, cache->v_page_stride, cache->v_token_stride, cache->v_head_stride},
                             {*cache, scales->k_page_stride, scales->k_token_stride, scales->k_head_stride},
                             {*cache, scales->v_page_stride, scales->v_token_stride, scales->v_head_stride}};
  const uint8_t* const bases[4] = {a.cache.k, a.cache.v, a.scales.k, a.scales.v};
  const long long row[4] = {D_qk / 2, D_v / 2, D_qk / 16, D_v / 16};
  for (int i = 0; k && i < 4; ++i)
    if (!dims[i].apart(row[i])) return ZYFA_ERR_INVALID_ARG;
  st = set_rope(a, rope, D_qk, N, positions, position_stride);
  if (st != ZYFA_OK) return st;
  if (N > 0x7fffffffll) return ZYFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(H) + H_kv > (1 << 16)) return ZYFA_ERR_UNSUPPORTED;
  const long long strides[3] = {q_token_stride, k_token_stride, v_token_stride};
  for (long long s : strides) {
    if (s < 0) return ZYFA_ERR_INVALID_ARG;
    if (s > (1ll << 40)) return ZYFA_ERR_UNSUPPORTED;
    if (s % 8 != 0) return ZYFA_ERR_MISALIGNED;
  }
  if (N == 0) return ZYFA_OK;
  if (!slots || (q && !q_out)) return ZYFA_ERR_INVALID_ARG;
  const void* rows[6] = {q, k, v, q ? q_out : nullptr, k_out, v_out};
  for (const void* p : rows)
    if (!aligned(p, 16)) return ZYFA_ERR_MISALIGNED;
  if (!aligned(slots, 8) || !aligned(k_descale, 4) || !aligned(v_descale, 4)) return ZYFA_ERR_MISALIGNED;
  const long long heads[3] = {static_cast<long long>(H) * D_qk, static_cast<long long>(H_kv) * D_qk, static_cast<long long>(H_kv) * D_v};
  const zyfa::Span outs[3] = {{q ? q_out : nullptr, N * heads[0] * 2}, {k ? k_out : nullptr, N * heads[1] * 2}, {k ? v_out : nullptr, N * heads[2] * 2}};
  const void* ins[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (zyfa::overlap(outs[i], outs[j])) return ZYFA_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j)
      if (zyfa::overlap(outs[i], {ins[j], heads[j] * 2, N, strides[j] * 2})) return ZYFA_ERR_INVALID_ARG;
  }
  for (int i = 0; k && i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (dims[j].meets(dims[i], bases[i] - bases[j], row[j], row[i])) return ZYFA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZYFA_ERR_CUDA;
  a.status = zyfa::device_status_word(dev);
  if (!a.status) return ZYFA_ERR_CUDA;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.q_tok = q_token_stride;
  a.k_tok = k_token_stride;
  a.v_tok = v_token_stride;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = k ? static_cast<__nv_bfloat16*>(k_out) : nullptr;
  a.v_out = k ? static_cast<__nv_bfloat16*>(v_out) : nullptr;
  a.positions = positions;
  a.pos_stride = position_stride;
  a.slots = slots;
  a.k_desc = k_descale;
  a.v_desc = v_descale;
  a.desc_per_head = descale_per_kv_head;
  a.N = N;
  a.H = H;
  const bool interleaved = rope && rope->interleaved, neat = a.offset % 16 == 0 && (interleaved || a.rot % 32 == 0);
  const cudaError_t e = interleaved ? launch<true>(a, neat, D_qk, dev, stream) : launch<false>(a, neat, D_qk, dev, stream);
  return e == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}
