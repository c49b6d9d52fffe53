// The page plan of a serving step: pages, slots and positions of the step's tokens from request lengths.
//
// Request b holds c_b tokens and adds n_b.  It starts need_b = ceil((c_b + n_b) / P) - ceil(c_b / P) pages,
// which are free_pages[cursor + sum_{a<b} need_a ...]; its token rows begin at cu_b = sum_{a<b} n_a.  Token i
// has position c_b + i, and slot page * P + position % P, where the page is a fresh one or the one of the
// table that the last cached token lies in.
//
// Bound: latency (the tables of a step are a few KB to a MB): 2.4 us for one request, 3.1 us for 256 with one token each
// and 3.1 us for 96 with 48 prompt chunks of up to 2048 tokens (on the GPU, in captured graphs), of which an empty launch is about 2 us.  (One block with a barrier
// per chunk of rows: 337 us for the 256.)  One launch: every block takes a run of token rows,
// forms the two prefix sums over the requests itself (1024 requests at a time in shared memory; the lengths come from
// L2 once another block has read them) rather than wait for another block, and finds the request of a row by
// bisection.  A fresh page always begins with a new token, so the thread of that token's row writes the table entry (the last
// block those of tokens that have no row) and no block depends on another's writes.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "paged.cuh"

namespace {

constexpr int kThreads = 256, kPerThread = 4, kChunk = kThreads * kPerThread, kWarps = kThreads / 32;

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
  int rows;             // token rows per block
  int cursor_only;      // a second launch that only moves the cursor
  int write_cursor;
  uint32_t page_magic;  // floor(t / page) = t * page_magic >> page_shift for t < 2^31
  int page_shift;
};

__device__ __forceinline__ int saturated(long long x) { return x > 0x7fffffffll ? 0x7fffffff : static_cast<int>(x); }

__global__ void __launch_bounds__(kThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ long long s_tok[kChunk + 1], s_page[kChunk];  // exclusive sums of n and need within the chunk
  __shared__ int s_cached[kChunk];
  __shared__ long long s_wtok[kWarps], s_wpage[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = blockIdx.x == 0 && !a.cursor_only;      // writes the per-request results
  const bool tail = blockIdx.x == gridDim.x - 1;            // takes the pages that tokens behind max_tokens start, too
  zyfa::wait_for_predecessor();
  const int cursor = max(0, *a.cursor_in);
  const int cap = a.max_pages * a.page;                     // at most 2^30
  const long long r0 = static_cast<long long>(blockIdx.x) * a.rows;
  const long long r1 = min(r0 + a.rows, static_cast<long long>(a.max_tokens));
  auto pages_before = [&](long long t) {                    // floor(t / page) of t <= cap + page
    return static_cast<int>((static_cast<unsigned long long>(t) * a.page_magic) >> a.page_shift);
  };
  long long tok = 0, page = 0;                              // sums over the chunks so far
  bool bad = false;
  for (int b0 = 0; b0 < a.B; b0 += kChunk) {
    // per-thread sums over its four requests, then across the warp and the block
    long long n[kPerThread], need[kPerThread], nsum = 0, psum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = b0 + tid * kPerThread + i;
      const int c = b < a.B ? max(0, a.cached[b]) : 0;
      n[i] = b < a.B ? max(0, a.fresh[b]) : 0;
      const long long len = c + n[i];
      const int had = pages_before(min(c, cap) + a.page - 1), has = pages_before(min(len, static_cast<long long>(cap)) + a.page - 1);
      need[i] = has - had;
      if (b < a.B) {
        s_cached[tid * kPerThread + i] = c;
        if (lead) {
          a.seq_lens[b] = static_cast<int>(min(len, static_cast<long long>(cap)));
          bad |= len > cap;
        }
      }
      nsum += n[i];
      psum += need[i];
    }
    long long ntok = nsum, npage = psum;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, ntok, s), v = __shfl_up_sync(0xffffffffu, npage, s);
      if (lane >= s) {
        ntok += u;
        npage += v;
      }
    }
    if (lane == 31) {
      s_wtok[warp] = ntok;
      s_wpage[warp] = npage;
    }
    __syncthreads();
    long long all_tok = 0, all_page = 0;
    ntok -= nsum;
    npage -= psum;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) {
        ntok += s_wtok[i];
        npage += s_wpage[i];
      }
      all_tok += s_wtok[i];
      all_page += s_wpage[i];
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int x = tid * kPerThread + i;
      s_tok[x] = ntok;
      s_page[x] = npage;
      if (lead && b0 + x < a.B) a.cu_tokens[b0 + x] = saturated(tok + ntok);
      ntok += n[i];
      npage += need[i];
    }
    if (tid == 0) s_tok[kChunk] = all_tok;
    __syncthreads();
    // this block's rows among the chunk's
    const long long end = a.cursor_only ? 0 : min(r1, tok + all_tok);
    for (long long r = max(r0, tok) + tid; r < end; r += kThreads) {
      const long long x = r - tok;
      int lo = 0, hi = min(kChunk, a.B - b0);               // s_tok[lo] <= x < s_tok[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tok[mid] <= x) lo = mid; else hi = mid;
      }
      const int c = s_cached[lo];
      const long long pos = c + (x - s_tok[lo]);
      long long slot = -1;
      if (pos < cap) {
        const int p = pages_before(pos), had = pages_before(min(c, cap) + a.page - 1), off = static_cast<int>(pos) - p * a.page;
        int* entry = a.table + static_cast<long long>(b0 + lo) * a.table_stride + p;
        int pg;
        if (p < had) {
          pg = *entry;
        } else {
          const long long f = cursor + page + s_page[lo] + (p - had);
          pg = f < a.num_free ? a.free_pages[f] : -1;
          if (off == 0) *entry = pg;
        }
        bad |= pg < 0;
        if (pg >= 0) slot = static_cast<long long>(pg) * a.page + off;
      }
      a.positions[r] = saturated(pos);
      a.slots[r] = slot;
    }
    // Tokens behind max_tokens are dropped, not the pages that they start.  (Page by page: lengths may name 2^31 tokens a request.)
    if (tail && !a.cursor_only && tok + all_tok > a.max_tokens) {
      for (long long x = tid; x < all_page; x += kThreads) {
        int lo = 0, hi = min(kChunk, a.B - b0);             // s_page[lo] <= x < s_page[hi]
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_page[mid] <= x) lo = mid; else hi = mid;
        }
        const int c = s_cached[lo], p = pages_before(min(c, cap) + a.page - 1) + static_cast<int>(x - s_page[lo]);
        if (tok + s_tok[lo] + static_cast<long long>(p) * a.page - c < a.max_tokens) continue;  // written with its first token's row
        const long long f = cursor + page + x;
        a.table[static_cast<long long>(b0 + lo) * a.table_stride + p] = f < a.num_free ? a.free_pages[f] : -1;
      }
    }
    tok += all_tok;
    page += all_page;
    __syncthreads();
  }
  for (long long r = max(r0, tok) + tid; r < r1 && !a.cursor_only; r += kThreads) {
    a.positions[r] = 0;
    a.slots[r] = -1;
  }
  if (lead && tid == 0) {
    a.cu_tokens[a.B] = saturated(tok);
    bad |= tok > a.max_tokens;
  }
  if (bad) atomicOr(a.status, zyfa::kStatusCapacityBit);
  if (tail && a.write_cursor && tid == 0)
    *a.cursor_out = static_cast<int>(min(cursor + page, static_cast<long long>(max(a.num_free, cursor))));
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
  // Every block reads the lengths, the pool and the table, at its own time.  (Of the cursors, which may be one, see below.)
  const long long n = B;
  const zyfa::Span outs[5] = {{seq_lens, n * 4}, {cu_tokens, n * 4 + 4}, {positions, max_tokens * 4ll}, {slots, max_tokens * 8ll}, {cursor_out, 4}};
  const zyfa::Span ins[5] = {{cached_lens, n * 4}, {new_lens, n * 4}, {free_pages, num_free * 4ll}, {block_table, max_pages * 4ll, n, table_stride * 4},
                             {cursor_in != cursor_out ? cursor_in : nullptr, 4}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (zyfa::overlap(outs[i], outs[j])) return ZYFA_ERR_INVALID_ARG;
    for (const zyfa::Span& x : ins)
      if (zyfa::overlap(outs[i], x)) return ZYFA_ERR_INVALID_ARG;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ZYFA_ERR_CUDA;
  int* status = zyfa::device_status_word(dev);
  if (!status) return ZYFA_ERR_CUDA;
  PlanArgs a = {};
  a.cached = cached_lens;
  a.fresh = new_lens;
  a.table = block_table;
  a.free_pages = free_pages;
  a.cursor_in = cursor_in;
  a.cursor_out = cursor_out;
  a.seq_lens = seq_lens;
  a.cu_tokens = cu_tokens;
  a.positions = positions;
  a.slots = slots;
  a.status = status;
  a.table_stride = table_stride;
  a.B = B;
  a.page = page_size;
  a.max_pages = max_pages;
  a.num_free = num_free;
  a.max_tokens = max_tokens;
  // t / page_size for t < 2^31: with s = ceil(log2 page_size) and M = floor(2^(31+s) / page_size) + 1 the error of
  // t M / 2^(31+s) is below 1 / page_size
  int s = 0;
  while ((1 << s) < page_size) ++s;
  a.page_shift = 31 + s;
  a.page_magic = static_cast<uint32_t>((1ull << (31 + s)) / static_cast<unsigned>(page_size) + 1);
  // One row per thread until the blocks fill the GPU several times over, then longer runs: each block repeats the sums.
  const long long most = 8ll * std::max(1, zyfa::device_sm_count(dev));
  const long long blocks = std::max(1ll, std::min(most, (max_tokens + kThreads - 1ll) / kThreads));
  a.rows = static_cast<int>((max_tokens + blocks - 1) / blocks);
  // Updated in place, the cursor may only be written once every block has read it.
  a.write_cursor = cursor_in != cursor_out || blocks == 1;
  if (zyfa::launch_dependent(plan_kernel, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, a) != cudaSuccess) return ZYFA_ERR_CUDA;
  if (!a.write_cursor) {
    a.write_cursor = a.cursor_only = 1;
    if (zyfa::launch_dependent(plan_kernel, dim3(1), kThreads, 0, stream, a) != cudaSuccess) return ZYFA_ERR_CUDA;
  }
  return ZYFA_OK;
}
