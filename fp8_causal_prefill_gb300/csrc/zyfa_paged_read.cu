// Tokens of a paged cache as dense rows: the other direction of the store, for prompts whose beginning is cached.
//
// Row n is token starts[b] + n - cu[b] of the request b whose run of rows n lies in.  A block takes some rows: it finds their requests
// (the run starts, or samples of them, searched in shared memory), then their pages, then writes whole passes of its threads; a thread
// keeps its 16 channels of a head (8 bytes of codes and a scale) while rows pass, so that where to read is an addition a row, has kBatch
// loads on their way, and stores 32 bytes of bf16 at once, two lines a quarter warp.  Bound by the memory: 131072 tokens of 8 heads of 128
// channels from 4 bits to bf16 in 105 to 106 us, 96% of what their bytes take (150 us with places found a piece at a time and 16-byte stores).
// Rows of e4m3 move half the bytes by as many loads and stores: 32768 tokens in 21.3 us, 73%.
//
// A value is x * f rounded once, with x = code * scale (6 bits for 4-bit caches, exact in fp16) and f = descale * fl(1 / out descale).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "paged.cuh"

namespace {

constexpr int kMaxRows = 128;  // rows per block at most
constexpr int kBatch = 4;      // of a thread's pieces on their way

struct ReadArgs {
  zyfa::CacheView cache;
  zyfa::ScaleView scales;
  const int* table;
  const int* cu;
  const int* starts;
  uint8_t *k_out, *v_out;
  const float *k_desc, *v_desc, *k_out_desc, *v_out_desc;
  int* status;
  long long table_stride, N, max_len;
  int B, rows;  // rows per block
  int wide;     // bf16 rows are aligned to 32 bytes
  int desc_per_head, desc_request, out_per_head;
  uint32_t page_magic;
  int page_shift;
  int step;  // from a sample of cu to the next
};

constexpr int kReadThreads = 256;

// What a thread reads of a head: 16 values of a cache type, and their scale.
template <int KIND>
struct Piece {
  static constexpr int kBytes = KIND == ZYFA_DTYPE_E2M1 ? 8 : KIND == ZYFA_DTYPE_E4M3 ? 16 : 32;
  static constexpr int kWords = kBytes / 4;
  uint32_t w[kWords], scale;
  __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* s) {
    if constexpr (KIND == ZYFA_DTYPE_E2M1) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x;
      w[1] = x.y;
      scale = *s;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 4 * i);
        w[i] = x.x;
        w[i + 1] = x.y;
        w[i + 2] = x.z;
        w[i + 3] = x.w;
      }
    }
  }
  static __device__ __forceinline__ void two(uint32_t f16, float* y) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f16));
    y[0] = v.x;
    y[1] = v.y;
  }
  // the values over their descale
  __device__ __forceinline__ void values(float (&y)[16]) const {
    if constexpr (KIND == ZYFA_DTYPE_E2M1) {
      const uint32_t s = zyfa::widen_e4m3(scale * 0x101u);  // in both halves
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        two(zyfa::mul_f16x2(zyfa::widen_e2m1<0>(w[i]), s), y + 8 * i);
        two(zyfa::mul_f16x2(zyfa::widen_e2m1<1>(w[i]), s), y + 8 * i + 2);
        two(zyfa::mul_f16x2(zyfa::widen_e2m1<2>(w[i]), s), y + 8 * i + 4);
        two(zyfa::mul_f16x2(zyfa::widen_e2m1<3>(w[i]), s), y + 8 * i + 6);
      }
    } else if constexpr (KIND == ZYFA_DTYPE_E4M3) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        two(zyfa::widen_e4m3(w[i]), y + 4 * i);
        two(zyfa::widen_e4m3_hi(w[i]), y + 4 * i + 2);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        y[2 * i] = __uint_as_float(w[i] << 16);
        y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};

// 16 bytes, or 32, at once where the rows are aligned to them (`wide`).
template <bool OUT_FP8>
__device__ __forceinline__ void put_words(uint8_t* to, const uint32_t (&w)[OUT_FP8 ? 4 : 8], bool wide) {
  if (OUT_FP8 || !wide) {
#pragma unroll
    for (int i = 0; i < (OUT_FP8 ? 4 : 8); i += 4) reinterpret_cast<uint4*>(to)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else if constexpr (!OUT_FP8) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                 "r"(w[6]), "r"(w[7])
                 : "memory");
  }
}

template <bool OUT_FP8>
__device__ __forceinline__ void put(uint8_t* to, const float (&y)[16], float f, bool wide) {
  constexpr int kWords = OUT_FP8 ? 4 : 8;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (OUT_FP8) {
      const float2 lo = zyfa::times(y[4 * i], y[4 * i + 1], f), hi = zyfa::times(y[4 * i + 2], y[4 * i + 3], f);
      asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
          "mov.b32 %0, {lo, hi};\n\t}"
          : "=r"(w[i])
          : "f"(lo.x), "f"(lo.y), "f"(hi.x), "f"(hi.y));
    } else {
      const float2 x = zyfa::times(y[2 * i], y[2 * i + 1], f);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x.y), "f"(x.x));
    }
  }
  put_words<OUT_FP8>(to, w, wide);
}

// Where a block's rows are: request (-2: none's, left as it is; -1: no page, zeros), and the token's bytes in the cache and in the scales.
struct Places {
  long long row[2][kMaxRows], scales[2][kMaxRows];  // K, V
  int request[kMaxRows];
};

// K (WHICH 0) or V (1) of the block's rows.  A thread keeps its 16 channels of a head while rows pass, several rows of few heads at a time.
template <int WHICH, int KIND, bool OUT_FP8, int D, int THREADS>
__device__ __forceinline__ void copy_rows(const ReadArgs& a, const Places& at, long long n0, int here) {
  constexpr int kPieces = D / 16, kOut = 16 * (OUT_FP8 ? 1 : 2);
  using P = Piece<KIND>;
  const int H_kv = a.cache.H_kv, all = H_kv * kPieces;
  const uint8_t *cache = WHICH ? a.cache.v : a.cache.k, *scales = WHICH ? a.scales.v : a.scales.k;
  const long long head_stride = WHICH ? a.cache.v_head : a.cache.k_head, scale_stride = WHICH ? a.scales.v_head : a.scales.k_head;
  const float *desc = WHICH ? a.v_desc : a.k_desc, *out_desc = WHICH ? a.v_out_desc : a.k_out_desc;
  uint8_t* const out = WHICH ? a.v_out : a.k_out;
  if (!out) return;
  const int step = all < THREADS ? THREADS / all : 1, first = all < THREADS ? static_cast<int>(threadIdx.x) / all : 0;
  if (first >= step) return;
  for (int item = threadIdx.x - first * all; item < all; item += THREADS) {
    const int h = item / kPieces, c = item % kPieces;
    const uint8_t* from = cache + h * head_stride + c * P::kBytes;
    const uint8_t* from_scales = scales + h * scale_stride + c;
    uint8_t* to = out + ((n0 + first) * all + item) * kOut;
    float inv = 1.0f, f = 1.0f;
    if (OUT_FP8 && out_desc) inv = __frcp_rn(out_desc[a.out_per_head ? h : 0]);
    const bool by_request = KIND != ZYFA_DTYPE_BF16 && desc && a.desc_request;
    if (KIND != ZYFA_DTYPE_BF16 && desc && !by_request) f = desc[a.desc_per_head ? h : 0];
    f *= inv;
    for (int r0 = first; r0 < here; r0 += kBatch * step) {
      P p[kBatch];
      int request[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * step;
        request[i] = r < here ? at.request[r] : -2;
        if (request[i] >= 0) p[i].load(from + at.row[WHICH][r], KIND == ZYFA_DTYPE_E2M1 ? from_scales + at.scales[WHICH][r] : nullptr);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (request[i] >= 0) {
          if (by_request) f = desc[static_cast<long long>(request[i]) * a.desc_request + h] * inv;
          float y[16];
          p[i].values(y);
          put<OUT_FP8>(to, y, f, a.wide);
        } else if (request[i] == -1) {
          const uint32_t none[OUT_FP8 ? 4 : 8] = {};
          put_words<OUT_FP8>(to, none, a.wide);
        }
        to += static_cast<long long>(step) * all * kOut;
      }
    }
  }
}

template <int KIND, bool OUT_FP8, int DQK, int DV>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kN = kReadThreads;
  __shared__ int s_cu[kN];
  __shared__ Places s_at;
  const int tid = threadIdx.x;
  const long long n0 = static_cast<long long>(blockIdx.x) * a.rows;
  const int here = static_cast<int>(min(static_cast<long long>(a.rows), a.N - n0));
  zyfa::wait_for_predecessor();
  // run starts: all of them, or every step-th
  const int samples = (a.B + a.step - 1) / a.step;
  if (tid < samples) s_cu[tid] = a.cu[tid * a.step];
  __syncthreads();
  if (tid < here) {
    const long long n = n0 + tid;
    int request = -2, off = 0;
    long long page = 0;
    if (n >= s_cu[0]) {
      int lo = 0, hi = samples;  // s_cu[lo] <= n, and the last such
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= n) lo = mid; else hi = mid;
      }
      int b = lo * a.step, end = min(a.B, b + a.step);
      while (end - b > 1) {
        const int mid = (b + end) >> 1;
        if (a.cu[mid] <= n) b = mid; else end = mid;
      }
      const long long first = a.cu[b];
      if (n < a.cu[b + 1] && n >= first) {
        const long long t = n - first + (a.starts ? a.starts[b] : 0);
        request = -1;
        if (t >= 0 && t < a.max_len) {
          const int p = static_cast<int>((static_cast<unsigned long long>(t) * a.page_magic) >> a.page_shift);
          page = a.table[b * a.table_stride + p];
          off = static_cast<int>(t - static_cast<long long>(p) * a.cache.page_size);
          if (page >= 0 && page < a.cache.num_pages) request = b;
        }
        if (request < 0) atomicOr(a.status, zyfa::kStatusBadPageBit);
      }
    }
    const zyfa::CacheView& c = a.cache;
    const zyfa::ScaleView& s = a.scales;
    s_at.row[0][tid] = page * c.k_page + off * c.k_tok;
    s_at.row[1][tid] = page * c.v_page + off * c.v_tok;
    s_at.scales[0][tid] = page * s.k_page + off * s.k_tok;
    s_at.scales[1][tid] = page * s.v_page + off * s.v_tok;
    s_at.request[tid] = request;
  }
  __syncthreads();
  copy_rows<0, KIND, OUT_FP8, DQK, kN>(a, s_at, n0, here);
  copy_rows<1, KIND, OUT_FP8, DV, kN>(a, s_at, n0, here);
}

template <int KIND, bool OUT_FP8>
cudaError_t launch(const ReadArgs& a, int D_qk, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.N + a.rows - 1) / a.rows));
  if (D_qk == 64) return zyfa::launch_dependent(read_kernel<KIND, OUT_FP8, 64, 64>, grid, kReadThreads, 0, stream, a);
  if (D_qk == 128) return zyfa::launch_dependent(read_kernel<KIND, OUT_FP8, 128, 128>, grid, kReadThreads, 0, stream, a);
  return zyfa::launch_dependent(read_kernel<KIND, OUT_FP8, 192, 128>, grid, kReadThreads, 0, stream, a);
}

template <int KIND>
cudaError_t launch(const ReadArgs& a, bool out_fp8, int D_qk, cudaStream_t stream) {
  return out_fp8 ? launch<KIND, true>(a, D_qk, stream) : launch<KIND, false>(a, D_qk, stream);
}

// The bytes from a cache's first row to its last one's end, as one run; nothing written may lie among them.
zyfa::Span extent(const void* base, const zyfa_paged_cache_t& c, long long page, long long tok, long long head, long long row) {
  const long double end = static_cast<long double>(c.num_pages - 1) * page + static_cast<long double>(c.page_size - 1) * tok +
                          static_cast<long double>(c.H_kv - 1) * head + row;
  return {base, static_cast<long long>(std::min<long double>(end, static_cast<long double>(1ll << 60)))};
}

}  // namespace

extern "C" zyfa_status_t zyfa_paged_read(const zyfa_paged_cache_t* cache, const zyfa_paged_scales_t* scales, const int* block_table,
                                         long long table_stride, int max_pages, const int* cu_tokens, const int* starts, int B,
                                         void* k_out, void* v_out, long long N, zyfa_dtype_t out_dtype, const float* k_descale,
                                         const float* v_descale, int descale_per_kv_head, const float* k_out_descale,
                                         const float* v_out_descale, int out_descale_per_kv_head, cudaStream_t stream) {
  using zyfa::aligned;
  ReadArgs a = {};
  zyfa_status_t st = zyfa::check_cache(cache, &a.cache, zyfa::kWideCaches | zyfa::k4BitCaches);
  if (st != ZYFA_OK) return st;
  const bool four = cache->dtype == ZYFA_DTYPE_E2M1;
  if (four != (scales != nullptr)) return ZYFA_ERR_INVALID_ARG;
  if (four) st = zyfa::check_scales(scales, &a.scales);
  if (st != ZYFA_OK) return st;
  if (out_dtype != ZYFA_DTYPE_E4M3 && out_dtype != ZYFA_DTYPE_BF16) return ZYFA_ERR_INVALID_ARG;
  if (B < 0 || N < 0 || max_pages < 0 || table_stride < max_pages) return ZYFA_ERR_INVALID_ARG;
  if (descale_per_kv_head != 0 && descale_per_kv_head != 1 && descale_per_kv_head != 3) return ZYFA_ERR_INVALID_ARG;
  if (out_descale_per_kv_head != 0 && out_descale_per_kv_head != 1) return ZYFA_ERR_INVALID_ARG;
  a.max_len = static_cast<long long>(max_pages) * cache->page_size;
  if (a.max_len > (1ll << 30) || B > 65536 || N > 0x7fffffffll || cache->H_kv > 65536) return ZYFA_ERR_UNSUPPORTED;
  if (N == 0 || B == 0) return ZYFA_OK;
  if ((!k_out && !v_out) || !cu_tokens || (max_pages > 0 && !block_table)) return ZYFA_ERR_INVALID_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return ZYFA_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(block_table), static_cast<const void*>(cu_tokens), static_cast<const void*>(starts),
                        static_cast<const void*>(k_descale), static_cast<const void*>(v_descale), static_cast<const void*>(k_out_descale),
                        static_cast<const void*>(v_out_descale)})
    if (!aligned(p, 4)) return ZYFA_ERR_MISALIGNED;
  const long long es = zyfa::element_size(out_dtype), heads = cache->H_kv, unit = zyfa::element_size(cache->dtype);
  const zyfa::Span outs[2] = {{k_out, N * heads * cache->D_qk * es}, {v_out, N * heads * cache->D_v * es}};
  const zyfa_paged_cache_t& c = *cache;
  const zyfa::Span ins[11] = {
      {block_table, max_pages * 4ll, B, table_stride * 4}, {cu_tokens, (B + 1) * 4ll}, {starts, B * 4ll},
      {k_descale, descale_per_kv_head == 1 ? B * heads * 4 : descale_per_kv_head ? heads * 4 : 4},
      {v_descale, descale_per_kv_head == 1 ? B * heads * 4 : descale_per_kv_head ? heads * 4 : 4},
      {k_out_descale, out_descale_per_kv_head ? heads * 4 : 4}, {v_out_descale, out_descale_per_kv_head ? heads * 4 : 4},
      extent(c.k, c, c.k_page_stride * unit, c.k_token_stride * unit, c.k_head_stride * unit, zyfa::row_bytes(c.dtype, c.D_qk)),
      extent(c.v, c, c.v_page_stride * unit, c.v_token_stride * unit, c.v_head_stride * unit, zyfa::row_bytes(c.dtype, c.D_v)),
      four ? extent(scales->k, c, scales->k_page_stride, scales->k_token_stride, scales->k_head_stride, c.D_qk / 16) : zyfa::Span(nullptr, 0),
      four ? extent(scales->v, c, scales->v_page_stride, scales->v_token_stride, scales->v_head_stride, c.D_v / 16) : zyfa::Span(nullptr, 0)};
  if (zyfa::overlap(outs[0], outs[1])) return ZYFA_ERR_INVALID_ARG;
  for (const zyfa::Span& out : outs)
    for (const zyfa::Span& x : ins)
      if (zyfa::overlap(out, x)) return ZYFA_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZYFA_ERR_CUDA;
  a.status = zyfa::device_status_word(dev);
  const int nsm = zyfa::device_sm_count(dev);
  if (!a.status || nsm <= 0) return ZYFA_ERR_CUDA;
  a.table = block_table;
  a.table_stride = table_stride;
  a.cu = cu_tokens;
  a.starts = starts;
  a.B = B;
  a.k_out = static_cast<uint8_t*>(k_out);
  a.v_out = static_cast<uint8_t*>(v_out);
  a.N = N;
  a.wide = aligned(k_out, 32) && aligned(v_out, 32);
  const bool fp8 = out_dtype == ZYFA_DTYPE_E4M3;
  a.k_desc = k_descale;
  a.v_desc = v_descale;
  a.k_out_desc = k_out_descale;
  a.v_out_desc = v_out_descale;
  a.desc_per_head = descale_per_kv_head != 0;
  a.desc_request = descale_per_kv_head == 1 ? cache->H_kv : 0;
  a.out_per_head = out_descale_per_kv_head;
  zyfa::division_by(cache->page_size, 30, &a.page_magic, &a.page_shift);
  a.step = (B + kReadThreads - 1) / kReadThreads;
  // Rows of a block: whole passes of its threads, 64 KiB to write (96 in e4m3, where the start counts more), but blocks for every SM four
  // times over.  131072 tokens of 8 heads of 128 as bf16: 105.9 us, with 96 KiB 107.5; 32768 as e4m3 from 4 bits 21.3 with 96 KiB,
  // 23.4 with 64, from bf16 34.1 and 35.0, from e4m3 28.8 and 25.2.
  const long long bytes = heads * (cache->D_qk + cache->D_v) * es, pass = std::max(1ll, kReadThreads / std::max(1ll, heads * cache->D_qk / 16));
  const long long most = std::max(pass, (es == 2 ? 65536 : 98304) / bytes / pass * pass), wanted = (N + 4ll * nsm - 1) / (4ll * nsm);
  a.rows = static_cast<int>(std::min<long long>(kMaxRows, std::min(most, (wanted + pass - 1) / pass * pass)));
  cudaError_t e;
  if (four)
    e = launch<ZYFA_DTYPE_E2M1>(a, fp8, cache->D_qk, stream);
  else if (cache->dtype == ZYFA_DTYPE_E4M3)
    e = launch<ZYFA_DTYPE_E4M3>(a, fp8, cache->D_qk, stream);
  else
    e = launch<ZYFA_DTYPE_BF16>(a, fp8, cache->D_qk, stream);
  return e == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}
