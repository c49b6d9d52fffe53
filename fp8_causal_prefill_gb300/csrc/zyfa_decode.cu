// Attention of one new token per request over a paged key/value cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax (in units of log2):
//   x_j = a q.k_j,  m' = max(m, max_j x_j),  l' = l 2^(m-m') + sum_j 2^(x_j-m'),  O' = O 2^(m-m') + sum_j 2^(x_j-m') v_j
// and out = dv O / l, lse = ln2 (m + log2 l), with a = scale dq dk log2(e).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "paged.cuh"

namespace {

constexpr int kThreads = 128;

struct DecodeArgs {
  const uint8_t* q;
  long long q_batch;  // bytes
  zyfa::CacheView cache;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  __nv_bfloat16* out;
  float* lse;
  const float *q_desc, *k_desc, *v_desc;
  int* status;
  float scale_log2;
  int desc_per_head;
  int max_pages, B, H;
};

template <bool FP8>
__device__ __forceinline__ float value(const uint8_t* row, int d) {
  if constexpr (FP8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(row[d], __NV_E4M3);
    return __half2float(h);
  } else {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
  }
}

__device__ __forceinline__ float descale(const float* p, int per_head, int i) { return p ? p[per_head ? i : 0] : 1.0f; }

template <bool FP8, int DQK, int DV>
__global__ void __launch_bounds__(kThreads) decode_kernel(const DecodeArgs a) {
  constexpr int es = FP8 ? 1 : 2;
  __shared__ float s_q[DQK], s_p[kThreads];
  __shared__ long long s_off[kThreads];
  __shared__ float s_red[4];
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int H_kv = a.cache.H_kv, hk = h / (a.H / H_kv), tid = threadIdx.x;
  const int P = a.cache.page_size;
  const int len = max(0, min(a.seq_lens[b], a.max_pages * P));
  for (int d = tid; d < DQK; d += kThreads) s_q[d] = value<FP8>(a.q + b * a.q_batch + h * DQK * es, d);
  const int di = b * H_kv + hk;
  const float c = FP8 ? a.scale_log2 * descale(a.q_desc, a.desc_per_head, di) * descale(a.k_desc, a.desc_per_head, di)
                      : a.scale_log2;
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  bool bad = false;
  for (int t0 = 0; t0 < len; t0 += kThreads) {
    const int t = t0 + tid;
    float x = -INFINITY;
    long long off = -1;
    if (t < len) {
      const int pg = a.table[b * a.table_stride + t / P];
      if (pg >= 0 && pg < a.cache.num_pages) {
        const uint8_t* kr = a.cache.k + pg * a.cache.k_page + (t % P) * a.cache.k_tok + hk * a.cache.k_head;
        off = pg * a.cache.v_page + (t % P) * a.cache.v_tok + hk * a.cache.v_head;
        float s = 0.0f;
        for (int d = 0; d < DQK; ++d) s = fmaf(s_q[d], value<FP8>(kr, d), s);
        x = s * c;
      } else {
        bad = true;
      }
    }
    __syncthreads();
    float top = x;
    for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
    if ((tid & 31) == 0) s_red[tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.0f : mn;
    s_p[tid] = exp2f(x - ref);
    s_off[tid] = off;
    const float corr = exp2f(m - ref);
    m = mn;
    l *= corr;
    o *= corr;
    __syncthreads();
    for (int j = 0; j < kThreads; ++j) {
      const float p = s_p[j];
      l += p;
      if (s_off[j] >= 0 && tid < DV) o = fmaf(p, value<FP8>(a.cache.v + s_off[j], tid), o);
    }
    __syncthreads();
  }
  const float dv = FP8 ? descale(a.v_desc, a.desc_per_head, di) : 1.0f;
  if (tid < DV) a.out[(static_cast<long long>(b) * a.H + h) * DV + tid] = __float2bfloat16_rn(l > 0.0f ? o / l * dv : 0.0f);
  if (a.lse && tid == 0)
    a.lse[static_cast<long long>(b) * a.H + h] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  if (bad) atomicOr(a.status, zyfa::kStatusBadPageBit);
}

template <bool FP8, int DQK, int DV>
cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
  decode_kernel<FP8, DQK, DV><<<static_cast<unsigned>(a.B) * a.H, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

extern "C" {

size_t zyfa_attn_decode_paged_workspace_bytes(int B, int H, int H_kv, int D_v) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || (D_v != 64 && D_v != 128)) return 0;
  return 16;
}

zyfa_status_t zyfa_attn_decode_paged(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache,
                                     const int* block_table, long long table_stride, int max_pages,
                                     const int* seq_lens, void* out, float* lse, int B, int H, float softmax_scale,
                                     const float* q_descale, const float* k_descale, const float* v_descale,
                                     int descale_per_kv_head, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  using zyfa::aligned;
  DecodeArgs a = {};
  const zyfa_status_t st = zyfa::check_cache(cache, &a.cache);
  if (st != ZYFA_OK) return st;
  const int H_kv = cache->H_kv, D_qk = cache->D_qk, D_v = cache->D_v;
  const bool fp8 = cache->dtype == ZYFA_DTYPE_E4M3;
  const int es = zyfa::element_size(cache->dtype);
  if (B < 0 || H < 1 || H % H_kv != 0 || max_pages < 0 || table_stride < max_pages) return ZYFA_ERR_INVALID_ARG;
  if (descale_per_kv_head != 0 && descale_per_kv_head != 1) return ZYFA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || softmax_scale < 0.0f) return ZYFA_ERR_INVALID_ARG;
  if (q_batch_stride < 0) return ZYFA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * cache->page_size > (1ll << 30)) return ZYFA_ERR_UNSUPPORTED;
  if (B > 65536 || H > 65536 || static_cast<long long>(B) * H > (1ll << 24)) return ZYFA_ERR_UNSUPPORTED;
  if (q_batch_stride > (1ll << 40)) return ZYFA_ERR_UNSUPPORTED;
  if (B == 0) return ZYFA_OK;
  if (!q || !out || !seq_lens || (max_pages > 0 && !block_table)) return ZYFA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || (q_batch_stride * es) % 16 != 0 || !aligned(out, 16) || !aligned(seq_lens, 4) ||
      !aligned(block_table, 4) || !aligned(lse, 4) || !aligned(q_descale, 4) || !aligned(k_descale, 4) ||
      !aligned(v_descale, 4))
    return ZYFA_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < zyfa_attn_decode_paged_workspace_bytes(B, H, H_kv, D_v)) return ZYFA_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return ZYFA_ERR_MISALIGNED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZYFA_ERR_CUDA;
  a.status = zyfa::device_status_word(dev);
  if (!a.status) return ZYFA_ERR_CUDA;
  if (softmax_scale == 0.0f) softmax_scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(D_qk)));
  a.scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  a.q = static_cast<const uint8_t*>(q);
  a.q_batch = q_batch_stride * es;
  a.table = block_table;
  a.table_stride = table_stride;
  a.seq_lens = seq_lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.q_desc = q_descale;
  a.k_desc = k_descale;
  a.v_desc = v_descale;
  a.desc_per_head = descale_per_kv_head;
  a.max_pages = max_pages;
  a.B = B;
  a.H = H;
  cudaError_t e;
  if (fp8)
    e = D_qk == 64 ? launch<true, 64, 64>(a, stream)
                   : D_qk == 128 ? launch<true, 128, 128>(a, stream) : launch<true, 192, 128>(a, stream);
  else
    e = D_qk == 64 ? launch<false, 64, 64>(a, stream)
                   : D_qk == 128 ? launch<false, 128, 128>(a, stream) : launch<false, 192, 128>(a, stream);
  return e == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}

}  // extern "C"
