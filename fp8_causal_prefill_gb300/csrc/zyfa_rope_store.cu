// Rotary positions with several axes, fused with the store into the paged key/value cache.
//
// Pair i of a token turns by angle = position[axis(i)] * inv_freq[i].  Far positions need more than the 24
// bits of an fp32 product, so the angle is taken in turns as a 64-bit fixed-point fraction: inv_freq is an
// fp32 number m * 2^e, turns-per-position = m * 2^e / (2 pi) is formed once from the integer m and 2^66 / (2 pi)
// to within 2^-64 of a turn, and position * fraction mod 2^64 is the exact reduction.  Its top 32 bits,
// read as signed, are the angle in half turns within [-1, 1).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.cuh"

namespace {

constexpr int kThreads = 256;

struct StoreArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_tok, k_tok, v_tok;  // elements
  uint8_t *q_out, *k_out, *v_out;
  const int* positions;
  long long pos_stride;
  const long long* slots;
  const float* inv_freq;
  const float *q_desc, *k_desc, *v_desc;
  int* status;
  long long N;
  zyfa::CacheView cache;
  int H, D_qk, D_v;
  int rot, offset, axis_end[4];
  int desc_per_head;
};

// 2^64 * |f| / (2 pi) modulo 2^64, with f's sign.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t bits = __float_as_uint(f);
  const int e = static_cast<int>((bits >> 23) & 255u);
  const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const uint64_t kC = 11743562013128004906ull;  // round(2^66 / (2 pi))
  const uint64_t lo = m * kC, hi = __umul64hi(m, kC);
  const int right = 2 - ((e ? e : 1) - 150);  // the value is (hi:lo) * 2^-right
  uint64_t r;
  if (right <= 0)
    r = right > -64 ? lo << -right : 0;
  else if (right < 64)
    r = (lo >> right) | (hi << (64 - right));
  else
    r = right < 128 ? hi >> (right - 64) : 0;
  return (bits >> 31) ? 0 - r : r;
}

__device__ __forceinline__ void angle_sincos(uint64_t fraction, int position, float* s, float* c) {
  const uint64_t t = static_cast<uint64_t>(static_cast<long long>(position)) * fraction;
  const int half_turns = static_cast<int>((t + (1ull << 31)) >> 32);
  sincospif(static_cast<float>(half_turns) * 4.656612873077393e-10f, s, c);  // * 2^-31
}

template <bool FP8>
__device__ __forceinline__ void put(uint8_t* row, int d, float y, float inv) {
  if constexpr (FP8) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(y * inv));
    row[d] = static_cast<uint8_t>(r);
  } else {
    reinterpret_cast<__nv_bfloat16*>(row)[d] = __float2bfloat16_rn(y);
  }
}

__device__ __forceinline__ float inverse(const float* desc, int i) { return desc ? __frcp_rn(desc[i]) : 1.0f; }

template <bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) store_kernel(const StoreArgs a) {
  constexpr int es = FP8 ? 1 : 2;
  const long long n = blockIdx.x;
  const long long slot = a.slots[n];
  if (slot < 0) return;
  const int H_kv = a.cache.H_kv, group = a.H / H_kv;
  const long long page = slot / a.cache.page_size, off = slot % a.cache.page_size;
  const bool in_cache = page < a.cache.num_pages;
  if (!in_cache && a.k && threadIdx.x == 0) atomicOr(a.status, zyfa::kStatusBadPageBit);
  // queries and keys: pairs of channels (rotated ones, then the plain ones two by two)
  const int pairs = a.D_qk / 2, half = a.rot / 2;
  const int first = a.q ? 0 : a.H, last = a.k ? a.H + H_kv : a.H;
  for (int i = threadIdx.x; i < (last - first) * pairs; i += kThreads) {
    const int h = first + i / pairs, p = i % pairs;
    int d0, d1;
    float s = 0.0f, c = 1.0f;
    if (p < half) {
      d0 = a.offset + (INTERLEAVED ? 2 * p : p);
      d1 = a.offset + (INTERLEAVED ? 2 * p + 1 : p + half);
      const int axis = (p >= a.axis_end[0]) + (p >= a.axis_end[1]) + (p >= a.axis_end[2]);
      angle_sincos(turn_fraction(a.inv_freq[p]), a.positions[axis * a.pos_stride + n], &s, &c);
    } else {
      d0 = 2 * (p - half);
      if (d0 >= a.offset) d0 += a.rot;
      d1 = d0 + 1;
    }
    const bool is_q = h < a.H;
    const int hk = is_q ? h / group : h - a.H;
    const __nv_bfloat16* x = is_q ? a.q + n * a.q_tok + h * a.D_qk : a.k + n * a.k_tok + hk * a.D_qk;
    const float u = __bfloat162float(x[d0]), w = __bfloat162float(x[d1]);
    const float y0 = u * c - w * s, y1 = u * s + w * c;
    const float inv = FP8 ? inverse(is_q ? a.q_desc : a.k_desc, a.desc_per_head ? hk : 0) : 1.0f;
    if (is_q) {
      uint8_t* o = a.q_out + (n * a.H + h) * a.D_qk * es;
      put<FP8>(o, d0, y0, inv);
      put<FP8>(o, d1, y1, inv);
    } else {
      if (in_cache) {
        uint8_t* o = a.cache.k + page * a.cache.k_page + off * a.cache.k_tok + hk * a.cache.k_head;
        put<FP8>(o, d0, y0, inv);
        put<FP8>(o, d1, y1, inv);
      }
      if (a.k_out) {
        uint8_t* o = a.k_out + (n * H_kv + hk) * a.D_qk * es;
        put<FP8>(o, d0, y0, inv);
        put<FP8>(o, d1, y1, inv);
      }
    }
  }
  if (!a.k) return;
  for (int i = threadIdx.x; i < H_kv * a.D_v; i += kThreads) {
    const int hk = i / a.D_v, d = i % a.D_v;
    const float y = __bfloat162float(a.v[n * a.v_tok + i]);
    const float inv = FP8 ? inverse(a.v_desc, a.desc_per_head ? hk : 0) : 1.0f;
    if (in_cache) put<FP8>(a.cache.v + page * a.cache.v_page + off * a.cache.v_tok + hk * a.cache.v_head, d, y, inv);
    if (a.v_out) put<FP8>(a.v_out + (n * H_kv + hk) * a.D_v * es, d, y, inv);
  }
}

}  // namespace

extern "C" zyfa_status_t zyfa_rope_paged_store(const void* q, const void* k, const void* v, long long q_token_stride,
                                               long long k_token_stride, long long v_token_stride, void* q_out,
                                               void* k_out, void* v_out, const int* positions,
                                               long long position_stride, const long long* slots, long long N, int H,
                                               const zyfa_paged_cache_t* cache, const zyfa_rope_t* rope,
                                               const float* q_descale, const float* k_descale, const float* v_descale,
                                               int descale_per_kv_head, cudaStream_t stream) {
  using zyfa::aligned;
  StoreArgs a = {};
  const zyfa_status_t st = zyfa::check_cache(cache, &a.cache);
  if (st != ZYFA_OK) return st;
  const int H_kv = cache->H_kv, D_qk = cache->D_qk, D_v = cache->D_v;
  if (N < 0 || H < 1 || H % H_kv != 0 || (descale_per_kv_head != 0 && descale_per_kv_head != 1)) return ZYFA_ERR_INVALID_ARG;
  if (!k != !v || (!q && !k)) return ZYFA_ERR_INVALID_ARG;
  // the cache is written here: its rows must not overlap
  if (k) {
    const bool apart =
        (H_kv == 1 || (cache->k_head_stride >= D_qk && cache->v_head_stride >= D_v)) &&
        (cache->page_size == 1 || (cache->k_token_stride >= D_qk && cache->v_token_stride >= D_v)) &&
        (cache->num_pages == 1 || (cache->k_page_stride >= D_qk && cache->v_page_stride >= D_v));
    if (!apart) return ZYFA_ERR_INVALID_ARG;
  }
  if (rope && rope->rot_dim != 0) {
    const zyfa_rope_t& r = *rope;
    if (r.rot_dim < 0 || r.rot_dim % 16 != 0 || r.rot_offset < 0 || r.rot_offset % 8 != 0) return ZYFA_ERR_INVALID_ARG;
    if (r.rot_dim > D_qk || r.rot_offset > D_qk - r.rot_dim) return ZYFA_ERR_INVALID_ARG;
    if ((r.interleaved != 0 && r.interleaved != 1) || r.num_axes < 1 || r.num_axes > 4) return ZYFA_ERR_INVALID_ARG;
    int total = 0;
    for (int i = 0; i < 4; ++i) {
      if (i < r.num_axes) {
        if (r.axis_pairs[i] < 0 || r.axis_pairs[i] > r.rot_dim / 2) return ZYFA_ERR_INVALID_ARG;
        total += r.axis_pairs[i];
      }
      a.axis_end[i] = i < r.num_axes - 1 ? total : 1 << 30;
    }
    if (total != r.rot_dim / 2) return ZYFA_ERR_INVALID_ARG;
    if (N > 0 && (!r.inv_freq || !positions)) return ZYFA_ERR_INVALID_ARG;
    if (r.num_axes > 1 && position_stride < N) return ZYFA_ERR_INVALID_ARG;
    if (!aligned(r.inv_freq, 4) || !aligned(positions, 4)) return ZYFA_ERR_MISALIGNED;
    a.rot = r.rot_dim;
    a.offset = r.rot_offset;
    a.inv_freq = r.inv_freq;
  }
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
  if (!aligned(slots, 8) || !aligned(q_descale, 4) || !aligned(k_descale, 4) || !aligned(v_descale, 4))
    return ZYFA_ERR_MISALIGNED;
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
  a.q_out = static_cast<uint8_t*>(q_out);
  a.k_out = k ? static_cast<uint8_t*>(k_out) : nullptr;
  a.v_out = k ? static_cast<uint8_t*>(v_out) : nullptr;
  a.positions = positions;
  a.pos_stride = position_stride;
  a.slots = slots;
  const bool fp8 = cache->dtype == ZYFA_DTYPE_E4M3;
  a.q_desc = q_descale;
  a.k_desc = k_descale;
  a.v_desc = v_descale;
  a.desc_per_head = descale_per_kv_head;
  a.N = N;
  a.H = H;
  a.D_qk = D_qk;
  a.D_v = D_v;
  const unsigned grid = static_cast<unsigned>(N);
  const bool il = rope && rope->interleaved;
  if (fp8 && il)
    store_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
  else if (fp8)
    store_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
  else if (il)
    store_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
  else
    store_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}
