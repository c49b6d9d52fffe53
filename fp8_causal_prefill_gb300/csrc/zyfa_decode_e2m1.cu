// Single-token attention over a 4-bit paged cache: C entry points (argument checks) and instantiations.
#include "decode_e2m1.cuh"

using namespace zyfa::decode4;

namespace {

zyfa_status_t attend(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache, const zyfa_paged_scales_t* scales,
                     const int* block_table, long long table_stride, int max_pages, const int* seq_lens, void* out, float* lse, int B, int H,
                     float softmax_scale, const float* k_descale, const float* v_descale, int descale_per_kv_head, void* workspace,
                     size_t workspace_bytes, bool stalled, cudaStream_t stream) {
  Args a = {};
  zyfa_status_t st = set_sizes(&a, cache, max_pages, B, H, zyfa::k4BitCaches);
  if (st == ZYFA_OK) st = zyfa::check_scales(scales, &a.scales);
  if (st == ZYFA_OK) st = set_call(a, q, q_batch_stride, 2, cache, block_table, table_stride, max_pages, seq_lens, out, lse, softmax_scale, nullptr, k_descale,
                                   v_descale, descale_per_kv_head, workspace, workspace_bytes, stalled);
  if (st != ZYFA_OK || B == 0) return st;
  int dev = 0, nsm = 0;
  st = set_device(a, &dev, &nsm);
  if (st != ZYFA_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return cache->D_qk == 64    ? launch4<64, 64>(a, nsm, dev, ws, stream)
         : cache->D_qk == 128 ? launch4<128, 128>(a, nsm, dev, ws, stream)
                              : launch4<192, 128>(a, nsm, dev, ws, stream);
}

template <int DQK, int DV>
int launches4(Args& a, int sms) {
  int smem;
  if (!(a.group <= 8 ? plan4<DQK, DV, 1>(a, sms, &smem) : plan4<DQK, DV, 2>(a, sms, &smem))) return 0;
  return a.whole ? 1 : 2;
}

}  // namespace

extern "C" {

int zyfa_attn_decode_paged_e2m1_launches(const zyfa_paged_cache_t* cache, const zyfa_paged_scales_t* scales, int max_pages, int B, int H,
                                         int sms, int* boxes) {
  Args a = {};
  if (set_sizes(&a, cache, max_pages, B, H, zyfa::k4BitCaches) != ZYFA_OK || zyfa::check_scales(scales, &a.scales) != ZYFA_OK || B == 0 || sms < 0) return 0;
  int dev = 0;
  if (sms == 0 && (cudaGetDevice(&dev) != cudaSuccess || (sms = zyfa::device_sm_count(dev)) <= 0)) return 0;
  sms = std::min(sms, kMaxSms);
  const int n = cache->D_qk == 64    ? launches4<64, 64>(a, sms)
                : cache->D_qk == 128 ? launches4<128, 128>(a, sms)
                                     : launches4<192, 128>(a, sms);
  if (n > 0 && boxes) *boxes = a.boxes;
  return n;
}

zyfa_status_t zyfa_attn_decode_paged_e2m1(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache, const zyfa_paged_scales_t* scales,
                                          const int* block_table, long long table_stride, int max_pages, const int* seq_lens, void* out,
                                          float* lse, int B, int H, float softmax_scale, const float* k_descale, const float* v_descale,
                                          int descale_per_kv_head, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return attend(q, q_batch_stride, cache, scales, block_table, table_stride, max_pages, seq_lens, out, lse, B, H, softmax_scale, k_descale, v_descale,
                descale_per_kv_head, workspace, workspace_bytes, false, stream);
}

zyfa_status_t zyfa_selftest_stalled_decode_e2m1(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache,
                                                const zyfa_paged_scales_t* scales, const int* block_table, long long table_stride,
                                                int max_pages, const int* seq_lens, void* out, int B, int H, void* workspace,
                                                size_t workspace_bytes, cudaStream_t stream) {
  return attend(q, q_batch_stride, cache, scales, block_table, table_stride, max_pages, seq_lens, out, nullptr, B, H, 0.0f, nullptr, nullptr, 0,
                workspace, workspace_bytes, true, stream);
}

}  // extern "C"
