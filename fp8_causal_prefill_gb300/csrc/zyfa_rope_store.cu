// Rotary positions with several axes, fused with the store into the paged key/value cache.
//
// Pair i of a token turns by angle = position[axis(i)] * inv_freq[i].  Far positions need more than the 24
// bits of an fp32 product, so the angle is taken in turns as a 64-bit fixed-point fraction: inv_freq is an
// fp32 number m * 2^e, turns-per-position = m * 2^e / (2 pi) is formed once from the integer m and 2^66 / (2 pi),
// off by at most (1 + |inv_freq| / 4) 2^-64, and position * fraction mod 2^64 is the exact reduction.  Its top 32 bits,
// read as signed, are the angle in half turns within [-1, 1).
//
// Bound: HBM.  Each value is read once (bf16) and written once or twice (cache, dense copy).  A block takes a few
// tokens; its threads first form the tokens' cosines and sines, once per (token, pair), in shared memory, then walk over
// the tokens' heads.  A thread keeps its 16 channels of a head: two 16-byte loads whose channels pair up (8 channels and
// their partners half the rotated width away, or 16 neighbours), eight rotations in packed fp32 pairs, one or two 8- or
// 16-byte stores per half.  The next head's loads are in flight while one is computed.
//
// Measured: a prompt of 32768 tokens (32 query and 8 KV heads of 128, e4m3 cache and dense copies) 111 us, 6.0 TB/s read and
// written (0.88 of a copy's rate; 0.71 of the DRAM's cycles); 4099 tokens with three axes in bf16 (16 and 4 heads of 64) 5.6 us
// (4.5 TB/s); 1 token, or 128 of them with 16 heads of 192/128, 3.3 us: a launch and three trips to memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "paged.cuh"

namespace {

constexpr int kMaxTokens = 32;  // tokens per block at most

// A multiple of the 16-channel pieces of a key head and of a value head.
template <int DQK>
constexpr int kThreads = DQK == 192 ? 192 : 256;

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
  int H;
  int rot, offset, axis_end[4];
  int desc_per_head;
  int tokens;  // per block
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

__device__ __forceinline__ float inverse(const float* desc, int i) { return desc ? __frcp_rn(desc[i]) : 1.0f; }

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ void widen8(const uint4& x, float (&y)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(w[i] << 16);
    y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Eight neighbouring values in the cache's type, `d` channels into `row` (and `copy`, where given).
template <bool FP8>
__device__ __forceinline__ void put8(uint8_t* row, uint8_t* copy, int d, const float (&y)[8], float inv) {
  if constexpr (FP8) {
    const uint2 x = make_uint2(codes4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                               codes4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
    if (row) *reinterpret_cast<uint2*>(row + d) = x;
    if (copy) *reinterpret_cast<uint2*>(copy + d) = x;
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
    const uint4 x = make_uint4(w[0], w[1], w[2], w[3]);
    if (row) *reinterpret_cast<uint4*>(row + 2 * d) = x;
    if (copy) *reinterpret_cast<uint4*>(copy + 2 * d) = x;
  }
}

// (a, b) -> (a c - b s, a s + b c) for two pairs at once
__device__ __forceinline__ void rotate2(float& a0, float& a1, float& b0, float& b1, const float* c, const float* s) {
  asm("{\n\t.reg .b64 a, b, c, s, n, y, z;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tmov.b64 c, {%4, %5};\n\t"
      "mov.b64 s, {%6, %7};\n\tmov.b64 n, {%8, %9};\n\tmul.rn.f32x2 y, b, n;\n\tfma.rn.f32x2 y, a, c, y;\n\tmul.rn.f32x2 z, b, c;\n\t"
      "fma.rn.f32x2 z, a, s, z;\n\tmov.b64 {%0, %1}, y;\n\tmov.b64 {%2, %3}, z;\n\t}"
      : "+f"(a0), "+f"(a1), "+f"(b0), "+f"(b1)
      : "f"(c[0]), "f"(c[1]), "f"(s[0]), "f"(s[1]), "f"(-s[0]), "f"(-s[1]));
}

// A thread's walk over (token, head) with a stride of `lanes` heads.
struct Walk {
  int token, head, heads, lanes;
  __device__ __forceinline__ void settle() {
    while (head >= heads) {
      head -= heads;
      ++token;
    }
  }
};

template <bool FP8, bool INTERLEAVED, int DQK, int DV>
__global__ void __launch_bounds__(kThreads<DQK>) store_kernel(const __grid_constant__ StoreArgs a) {
  constexpr int es = FP8 ? 1 : 2, kN = kThreads<DQK>;
  constexpr int kPiecesK = DQK / 16, kPiecesV = DV / 16, kHalf = DQK / 2;
  static_assert(kN % kPiecesK == 0 && kN % kPiecesV == 0);
  __shared__ __align__(16) float s_cos[kMaxTokens][kHalf], s_sin[kMaxTokens][kHalf];
  __shared__ long long s_krow[kMaxTokens], s_vrow[kMaxTokens];  // offsets in the cache; -1: not written, -2: padding
  const int tid = threadIdx.x;
  const int tokens = a.tokens;
  const long long n0 = static_cast<long long>(blockIdx.x) * tokens;
  const int here = static_cast<int>(min(static_cast<long long>(tokens), a.N - n0));
  const int H_kv = a.cache.H_kv, half = a.rot / 2, heads_q = a.q ? a.H : 0;

  // queries and keys: this thread's 16 channels, the same of every head
  const int j = tid % kPiecesK;
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
  Walk w = {0, tid / kPiecesK, heads_q + (a.k ? H_kv : 0), kN / kPiecesK};
  w.settle();
  uint4 x0, x1;
  auto fetch = [&]() {
    if (w.token >= here) return;
    const long long n = n0 + w.token;
    const __nv_bfloat16* x = w.head < heads_q ? a.q + n * a.q_tok + w.head * DQK : a.k + n * a.k_tok + (w.head - heads_q) * DQK;
    x0 = *reinterpret_cast<const uint4*>(x + d0);
    x1 = *reinterpret_cast<const uint4*>(x + d1);
  };
  // values
  const int dv = tid % kPiecesV * 16;
  Walk wv = {0, tid / kPiecesV, H_kv, kN / kPiecesV};
  wv.settle();
  uint4 y0, y1;
  auto fetch_v = [&]() {
    if (wv.token >= here) return;
    const __nv_bfloat16* x = a.v + (n0 + wv.token) * a.v_tok + wv.head * DV + dv;
    y0 = *reinterpret_cast<const uint4*>(x);
    y1 = *reinterpret_cast<const uint4*>(x + 8);
  };
  zyfa::wait_for_predecessor();
  // the first loads run while the tables are made
  fetch();
  if (a.k) fetch_v();
  if (tid < here) {
    const long long slot = a.slots[n0 + tid];
    long long krow = -2, vrow = 0;
    if (slot >= 0) {
      long long page, off;
      if (slot <= 0x7fffffffll) {
        page = static_cast<unsigned>(slot) / static_cast<unsigned>(a.cache.page_size);
        off = static_cast<unsigned>(slot) % static_cast<unsigned>(a.cache.page_size);
      } else {
        page = slot / a.cache.page_size;
        off = slot % a.cache.page_size;
      }
      krow = -1;
      if (page < a.cache.num_pages) {
        krow = page * a.cache.k_page + off * a.cache.k_tok;
        vrow = page * a.cache.v_page + off * a.cache.v_tok;
      } else if (a.k) {
        atomicOr(a.status, zyfa::kStatusBadPageBit);
      }
    }
    s_krow[tid] = krow;
    s_vrow[tid] = vrow;
  }
  if (half > 0) {  // a thread keeps its pair: kN / half tokens at a time
    const int at_once = kN / half, t0 = tid / half, p = tid - t0 * half;
    if (t0 < min(at_once, here)) {
      const int axis = (p >= a.axis_end[0]) + (p >= a.axis_end[1]) + (p >= a.axis_end[2]);
      const int* position = a.positions + axis * a.pos_stride + n0;
      const float frequency = a.inv_freq[p];
      const uint64_t fraction = turn_fraction(frequency);
      const bool finite = isfinite(frequency);  // an infinity or NaN has no turns
      for (int t = t0; t < here; t += at_once) {
        float s, c;
        angle_sincos(fraction, position[t], &s, &c);
        s_sin[t][p] = finite ? s : NAN;
        s_cos[t][p] = finite ? c : NAN;
      }
    }
  }
  __syncthreads();
  const bool per_head = a.desc_per_head;
  const float q_inv = FP8 ? inverse(a.q_desc, 0) : 1.0f, k_inv = FP8 ? inverse(a.k_desc, 0) : 1.0f, v_inv = FP8 ? inverse(a.v_desc, 0) : 1.0f;

  while (a.k && wv.token < here) {
    const int token = wv.token, head = wv.head;
    float u[8], v[8];
    widen8(y0, u);
    widen8(y1, v);
    wv.head += wv.lanes;
    wv.settle();
    fetch_v();
    const long long krow = s_krow[token];
    if (krow == -2) continue;
    uint8_t* row = krow >= 0 ? a.cache.v + s_vrow[token] + head * a.cache.v_head : nullptr;
    uint8_t* copy = a.v_out ? a.v_out + ((n0 + token) * H_kv + head) * DV * es : nullptr;
    const float inv = FP8 && per_head ? inverse(a.v_desc, head) : v_inv;
    put8<FP8>(row, copy, dv, u, inv);
    put8<FP8>(row, copy, dv + 8, v, inv);
  }
  while (w.token < here) {
    const int token = w.token, head = w.head;
    float u[8], v[8];
    widen8(x0, u);
    widen8(x1, v);
    w.head += w.lanes;
    w.settle();
    fetch();
    const long long krow = s_krow[token];
    if (krow == -2) continue;
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
    uint8_t *row = nullptr, *copy = nullptr;
    float inv;
    if (head < heads_q) {
      row = a.q_out + (n * a.H + head) * DQK * es;
      inv = FP8 && per_head ? inverse(a.q_desc, head / (a.H / H_kv)) : q_inv;
    } else {
      const int hk = head - heads_q;
      if (krow >= 0) row = a.cache.k + krow + hk * a.cache.k_head;
      if (a.k_out) copy = a.k_out + (n * H_kv + hk) * DQK * es;
      inv = FP8 && per_head ? inverse(a.k_desc, hk) : k_inv;
    }
    put8<FP8>(row, copy, d0, u, inv);
    put8<FP8>(row, copy, d1, v, inv);
  }
}

template <bool FP8, bool INTERLEAVED>
cudaError_t launch(const StoreArgs& a, int D_qk, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.N + a.tokens - 1) / a.tokens);
  if (D_qk == 64)
    return zyfa::launch_dependent(store_kernel<FP8, INTERLEAVED, 64, 64>, dim3(grid), kThreads<64>, 0, stream, a);
  if (D_qk == 128)
    return zyfa::launch_dependent(store_kernel<FP8, INTERLEAVED, 128, 128>, dim3(grid), kThreads<128>, 0, stream, a);
  return zyfa::launch_dependent(store_kernel<FP8, INTERLEAVED, 192, 128>, dim3(grid), kThreads<192>, 0, stream, a);
}

// Where the rows of a cache begin: the sums of multiples, below their extents, of three strides (elements), the largest first.
struct CacheDims {
  long long extent[3], stride[3];
  CacheDims(const zyfa_paged_cache_t& c, long long page, long long token, long long head) {
    std::pair<long long, long long> d[3] = {{page, c.num_pages}, {token, c.page_size}, {head, c.H_kv}};
    for (auto& x : d)
      if (x.second == 1) x.first = 0;  // a stride that is never taken
    std::sort(d, d + 3);
    for (int i = 0; i < 3; ++i) {
      stride[i] = d[2 - i].first;
      extent[i] = d[2 - i].second;
    }
  }
  // The rows, of D elements, do not overlap: each stride passes over everything within it, as in any view of a dense tensor.
  // (Strides that miss one another by their remainders alone are refused.)
  bool apart(long long D) const {
    long long span = D;
    for (int i = 2; i >= 0; --i) {
      if (extent[i] == 1) continue;
      if (stride[i] < span) return false;
      if (stride[i] > (1ll << 60) / extent[i]) return i == 0;  // more than any memory, and nothing may lie around it
      span += (extent[i] - 1) * stride[i];
    }
    return true;
  }
  // A row of D elements of this cache and one of `other_D`, `offset` elements behind, overlap somewhere.  Decided for equal strides
  // (rows apart in both); with others, as of K and V blocks side by side within a page, the caller answers for them.
  bool meets(const CacheDims& other, long long offset, long long D, long long other_D) const {
    for (int i = 0; i < 3; ++i)
      if (stride[i] != other.stride[i] || extent[i] != other.extent[i]) return offset == 0;
    return meets_from(0, offset, D, other_D);
  }

 private:
  bool meets_from(int i, long long offset, long long D, long long other_D) const {
    if (i == 3) return offset < D && -offset < other_D;
    if (extent[i] == 1) return meets_from(i + 1, offset, D, other_D);
    // what is left has to lie within this stride
    long long n = offset / stride[i];
    if (offset % stride[i] < 0) --n;
    for (long long x : {n, n + 1})
      if (x > -extent[i] && x < extent[i] && meets_from(i + 1, offset - x * stride[i], D, other_D)) return true;
    return false;
  }
};

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
  const CacheDims kdims(*cache, cache->k_page_stride, cache->k_token_stride, cache->k_head_stride);
  const CacheDims vdims(*cache, cache->v_page_stride, cache->v_token_stride, cache->v_head_stride);
  if (k && !(kdims.apart(D_qk) && vdims.apart(D_v))) return ZYFA_ERR_INVALID_ARG;
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
  const long long es = zyfa::element_size(cache->dtype), heads[3] = {static_cast<long long>(H) * D_qk, static_cast<long long>(H_kv) * D_qk,
                                                                     static_cast<long long>(H_kv) * D_v};
  const zyfa::Span outs[3] = {{q ? q_out : nullptr, N * heads[0] * es}, {k ? k_out : nullptr, N * heads[1] * es}, {k ? v_out : nullptr, N * heads[2] * es}};
  const void* ins[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (zyfa::overlap(outs[i], outs[j])) return ZYFA_ERR_INVALID_ARG;
    for (int j = 0; j < 3; ++j)
      if (zyfa::overlap(outs[i], {ins[j], heads[j] * 2, N, strides[j] * 2})) return ZYFA_ERR_INVALID_ARG;
  }
  if (k && kdims.meets(vdims, (a.cache.v - a.cache.k) / zyfa::element_size(cache->dtype), D_qk, D_v)) return ZYFA_ERR_INVALID_ARG;
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
  // Several tokens per block share its start-up (its tables, 1 to 2 us of latency), few heads more than many; then as many as fill
  // whole waves of the blocks that the GPU holds (4 an SM of 256 threads, 6 of 192).  At most 8, 12 and 16 tokens, waves filled: 112.1,
  // 111.1 and 111.3 us for 32768 tokens (FP8, 32 + 8 heads of 128), 21.8, 20.0 and 17.0 for 19164 with 4 + 2 heads, 15.2 with 32;
  // 5031 tokens of 32 + 8 heads of 64 as 629 blocks of 8, a wave and a bit, 15.3 us, as 559 of 9 12.6.
  const long long slots_gpu = (D_qk == 192 ? 6ll : 4ll) * std::max(1, zyfa::device_sm_count(dev));
  const long long most = std::min(kMaxTokens, std::max(12, 320 / (H + 2 * H_kv)));
  const long long waves = (N + most * slots_gpu - 1) / (most * slots_gpu);
  a.tokens = static_cast<int>((N + slots_gpu * waves - 1) / (slots_gpu * waves));
  const bool il = rope && rope->interleaved;
  cudaError_t e;
  if (fp8)
    e = il ? launch<true, true>(a, D_qk, stream) : launch<true, false>(a, D_qk, stream);
  else
    e = il ? launch<false, true>(a, D_qk, stream) : launch<false, false>(a, D_qk, stream);
  return e == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}
