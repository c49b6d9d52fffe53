// The page plan of a serving step: pages, slots and positions of the step's tokens from request lengths.
//
// Request b holds c_b tokens and adds n_b.  It starts need_b = ceil((c_b + n_b) / P) - ceil(c_b / P) pages,
// which are free_pages[cursor + sum_{a<b} need_a ...]; its token rows begin at cu_b = sum_{a<b} n_a.  Token i
// has position c_b + i, and slot page * P + position % P, where the page is a fresh one or the one of the
// table that the last cached token lies in.
#include <cuda_runtime.h>

#include <cstdint>

#include "paged.cuh"

namespace {

constexpr int kThreads = 1024;

struct PlanArgs {
  const int* cached;
  const int* fresh;
  int* table;
  const int* free_pages;
  const int* cursor_in;
  int* cursor_out;
  int* seq_lens;
  int* cu_tokens;
  int* positions;
  long long* slots;
  int* status;
  long long table_stride;
  int B, page, max_pages, num_free, max_tokens;
};

__device__ __forceinline__ int saturated(long long x) { return x > 0x7fffffffll ? 0x7fffffff : static_cast<int>(x); }

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  __shared__ long long s_tok, s_page;
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  if (tid == 0) {
    s_tok = 0;
    s_page = 0;
    s_bad = 0;
  }
  __syncthreads();
  const long long cursor = max(0, *a.cursor_in);
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  for (int b = 0; b < a.B; ++b) {
    const long long c = max(0, a.cached[b]), n = max(0, a.fresh[b]);
    const long long len = c + n;
    const int had = static_cast<int>(min((c + a.page - 1) / a.page, static_cast<long long>(a.max_pages)));
    const int has = static_cast<int>(min((len + a.page - 1) / a.page, static_cast<long long>(a.max_pages)));
    const long long first = cursor + s_page, row = s_tok;
    int* table = a.table + b * a.table_stride;
    bool bad = len > cap || row + n > a.max_tokens;
    for (int p = had + tid; p < has; p += kThreads) {
      const long long f = first + p - had;
      table[p] = f < a.num_free ? a.free_pages[f] : -1;
      bad |= f >= a.num_free;
    }
    for (long long i = tid; i < n && row + i < a.max_tokens; i += kThreads) {
      const long long pos = c + i;
      long long slot = -1;
      if (pos < cap) {
        const int p = static_cast<int>(pos / a.page);
        const long long f = first + p - had;
        const int pg = p < had ? table[p] : f < a.num_free ? a.free_pages[f] : -1;
        if (pg >= 0) slot = static_cast<long long>(pg) * a.page + pos % a.page;
        bad |= pg < 0;
      }
      a.positions[row + i] = saturated(pos);
      a.slots[row + i] = slot;
    }
    if (bad) s_bad = 1;
    if (tid == 0) {
      a.seq_lens[b] = static_cast<int>(min(len, cap));
      a.cu_tokens[b] = saturated(row);
    }
    __syncthreads();
    if (tid == 0) {
      s_tok = row + n;
      s_page += has - had;
    }
    __syncthreads();
  }
  for (long long i = s_tok + tid; i < a.max_tokens; i += kThreads) {
    a.positions[i] = 0;
    a.slots[i] = -1;
  }
  if (tid == 0) {
    a.cu_tokens[a.B] = saturated(s_tok);
    *a.cursor_out = static_cast<int>(min(cursor + s_page, static_cast<long long>(max(a.num_free, static_cast<int>(cursor)))));
    if (s_bad) atomicOr(a.status, zyfa::kStatusCapacityBit);
  }
}

}  // namespace

extern "C" zyfa_status_t zyfa_paged_plan(const int* cached_lens, const int* new_lens, int B, int page_size,
                                         int* block_table, long long table_stride, int max_pages,
                                         const int* free_pages, int num_free, const int* cursor_in, int* cursor_out,
                                         int* seq_lens, int* cu_tokens, int* positions, long long* slots,
                                         int max_tokens, cudaStream_t stream) {
  using zyfa::aligned;
  if (B < 0 || max_tokens < 0 || num_free < 0 || max_pages < 0 || table_stride < max_pages) return ZYFA_ERR_INVALID_ARG;
  if (page_size < 1 || page_size > 65536) return ZYFA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * page_size > (1ll << 30) || B > 65536) return ZYFA_ERR_UNSUPPORTED;
  if (!cursor_in || !cursor_out || !cu_tokens) return ZYFA_ERR_INVALID_ARG;
  if (B > 0 && (!cached_lens || !new_lens || !seq_lens || (max_pages > 0 && !block_table))) return ZYFA_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_pages) || (max_tokens > 0 && (!positions || !slots))) return ZYFA_ERR_INVALID_ARG;
  const void* ints[9] = {cached_lens, new_lens, block_table, free_pages, cursor_in, cursor_out, seq_lens, cu_tokens,
                         positions};
  for (const void* p : ints)
    if (!aligned(p, 4)) return ZYFA_ERR_MISALIGNED;
  if (!aligned(slots, 8)) return ZYFA_ERR_MISALIGNED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZYFA_ERR_CUDA;
  int* status = zyfa::device_status_word(dev);
  if (!status) return ZYFA_ERR_CUDA;
  const PlanArgs a = {cached_lens, new_lens,  block_table, free_pages, cursor_in, cursor_out, seq_lens,   cu_tokens,
                      positions,   slots,     status,      table_stride, B,       page_size,  max_pages,  num_free,
                      max_tokens};
  plan_kernel<<<1, kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}
