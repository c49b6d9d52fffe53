// Single-token attention over a paged cache: C entry points (argument checks, page arithmetic).
#include "decode.cuh"

using namespace zyfa::decode;

namespace {

zyfa_status_t attend(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache, const int* block_table,
                     long long table_stride, int max_pages, const int* seq_lens, void* out, float* lse, int B, int H,
                     float softmax_scale, const float* q_descale, const float* k_descale, const float* v_descale,
                     int descale_per_kv_head, void* workspace, size_t workspace_bytes, bool stalled, cudaStream_t stream) {
  DecodeArgs a = {};
  zyfa_status_t st = set_sizes(&a, cache, max_pages, B, H);
  if (st != ZYFA_OK) return st;
  const bool fp8 = cache->dtype == ZYFA_DTYPE_E4M3;
  st = set_call(a, q, q_batch_stride, zyfa::element_size(cache->dtype), cache, block_table, table_stride, max_pages, seq_lens, out, lse, softmax_scale,
                q_descale, k_descale, v_descale, descale_per_kv_head, workspace, workspace_bytes, stalled);
  int dev = 0, nsm = 0;
  if (st == ZYFA_OK && B > 0) st = set_device(a, &dev, &nsm);
  if (st != ZYFA_OK || B == 0) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return fp8 ? zyfa::decode_fp8(a, cache->D_qk, nsm, dev, ws, stream) : zyfa::decode_bf16(a, cache->D_qk, nsm, dev, ws, stream);
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
