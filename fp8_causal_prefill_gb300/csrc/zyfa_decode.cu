// Single-token attention over a paged cache: C entry points (argument checks, page arithmetic).
#include "decode.cuh"

using namespace zyfa::decode;

namespace {

// What the call's sizes decide, checked.
zyfa_status_t set_sizes(DecodeArgs* a, const zyfa_paged_cache_t* cache, int max_pages, int B, int H) {
  const zyfa_status_t st = zyfa::check_cache(cache, &a->cache);
  if (st != ZYFA_OK) return st;
  if (B < 0 || H < 1 || H % cache->H_kv != 0 || max_pages < 0) return ZYFA_ERR_INVALID_ARG;
  const long long max_len = static_cast<long long>(max_pages) * cache->page_size;
  if (max_len > (1ll << 30)) return ZYFA_ERR_UNSUPPORTED;
  if (B > 65536 || H > 65536 || static_cast<long long>(B) * H > (1ll << 24)) return ZYFA_ERR_UNSUPPORTED;
  // the schedule numbers tiles, and a gap behind each request, in 31 bits
  if (B * ((max_len + 15) / 16 + kGap) > 0x7fffffffll) return ZYFA_ERR_UNSUPPORTED;
  a->max_len = static_cast<int>(max_len);
  a->B = B;
  a->H = H;
  a->group = H / cache->H_kv;
  return ZYFA_OK;
}

zyfa_status_t attend(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache, const int* block_table,
                     long long table_stride, int max_pages, const int* seq_lens, void* out, float* lse, int B, int H,
                     float softmax_scale, const float* q_descale, const float* k_descale, const float* v_descale,
                     int descale_per_kv_head, void* workspace, size_t workspace_bytes, bool stalled, cudaStream_t stream) {
  using zyfa::aligned;
  DecodeArgs a = {};
  const zyfa_status_t st = set_sizes(&a, cache, max_pages, B, H);
  if (st != ZYFA_OK) return st;
  const int H_kv = cache->H_kv, D_qk = cache->D_qk, D_v = cache->D_v;
  const bool fp8 = cache->dtype == ZYFA_DTYPE_E4M3;
  const int es = zyfa::element_size(cache->dtype);
  if (table_stride < max_pages) return ZYFA_ERR_INVALID_ARG;
  if (descale_per_kv_head != 0 && descale_per_kv_head != 1 && descale_per_kv_head != 3) return ZYFA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || softmax_scale < 0.0f) return ZYFA_ERR_INVALID_ARG;
  if (q_batch_stride < 0) return ZYFA_ERR_INVALID_ARG;
  if (q_batch_stride > (1ll << 40)) return ZYFA_ERR_UNSUPPORTED;
  if (B == 0) return ZYFA_OK;
  if (!q || !out || !seq_lens || (max_pages > 0 && !block_table)) return ZYFA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || (q_batch_stride * es) % 16 != 0 || !aligned(out, 16) || !aligned(seq_lens, 4) ||
      !aligned(block_table, 4) || !aligned(lse, 4) || !aligned(q_descale, 4) || !aligned(k_descale, 4) ||
      !aligned(v_descale, 4))
    return ZYFA_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < zyfa_attn_decode_paged_workspace_bytes(B, H, H_kv, D_v, a.max_len))
    return ZYFA_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return ZYFA_ERR_MISALIGNED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ZYFA_ERR_CUDA;
  a.status = zyfa::device_status_word(dev);
  const int nsm = std::min(zyfa::device_sm_count(dev), kMaxSms);
  if (!a.status || nsm <= 0) return ZYFA_ERR_CUDA;
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
  a.desc_per_head = descale_per_kv_head != 0;
  a.desc_request = descale_per_kv_head == 1 ? H_kv : 0;
  // t / page_size for t < 2^30: with s = ceil(log2 page_size) and M = floor(2^(30+s) / page_size) + 1 the error of
  // t M / 2^(30+s) is below 1 / page_size
  int s = 0;
  while ((1 << s) < cache->page_size) ++s;
  a.page_shift = 30 + s;
  a.page_magic = static_cast<uint32_t>((1ull << (30 + s)) / static_cast<unsigned>(cache->page_size) + 1);
  a.wait_clocks = stalled ? kShortWaitClocks : kWaitClocks;
  a.stalled = stalled;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return fp8 ? zyfa::decode_fp8(a, D_qk, nsm, dev, ws, stream) : zyfa::decode_bf16(a, D_qk, nsm, dev, ws, stream);
}
}  // namespace

extern "C" {

size_t zyfa_attn_decode_paged_workspace_bytes(int B, int H, int H_kv, int D_v, long long max_len) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || (D_v != 64 && D_v != 128) || max_len < 0) return 0;
  const long long parts = parts_at_most(B, H, H_kv, max_len);
  return static_cast<size_t>(round_up((B + 2ll) * 4, 256) + round_up(2 * parts * H * 8, 256) + 2 * parts * H * D_v * 4);
}

int zyfa_attn_decode_paged_launches(const zyfa_paged_cache_t* cache, int max_pages, int B, int H, int sms) {
  DecodeArgs a = {};
  if (set_sizes(&a, cache, max_pages, B, H) != ZYFA_OK || B == 0 || sms < 0) return 0;
  int dev = 0;
  if (sms == 0 && (cudaGetDevice(&dev) != cudaSuccess || (sms = zyfa::device_sm_count(dev)) <= 0)) return 0;
  sms = std::min(sms, kMaxSms);
  return cache->dtype == ZYFA_DTYPE_E4M3 ? zyfa::decode_launches_fp8(a, cache->D_qk, sms) : zyfa::decode_launches_bf16(a, cache->D_qk, sms);
}

zyfa_status_t zyfa_attn_decode_paged(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache,
                                     const int* block_table, long long table_stride, int max_pages,
                                     const int* seq_lens, void* out, float* lse, int B, int H, float softmax_scale,
                                     const float* q_descale, const float* k_descale, const float* v_descale,
                                     int descale_per_kv_head, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  return attend(q, q_batch_stride, cache, block_table, table_stride, max_pages, seq_lens, out, lse, B, H, softmax_scale, q_descale,
                k_descale, v_descale, descale_per_kv_head, workspace, workspace_bytes, false, stream);
}

zyfa_status_t zyfa_selftest_stalled_decode(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache,
                                           const int* block_table, long long table_stride, int max_pages,
                                           const int* seq_lens, void* out, int B, int H, void* workspace,
                                           size_t workspace_bytes, cudaStream_t stream) {
  return attend(q, q_batch_stride, cache, block_table, table_stride, max_pages, seq_lens, out, nullptr, B, H, 0.0f, nullptr, nullptr,
                nullptr, 0, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
