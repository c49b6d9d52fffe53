// What the paged serving operators share: status bits, the device view of a paged cache, its host checks.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "zyfa.h"

namespace zyfa {

// Bits of the library's per-device status word (zyfa_check_errors clears and reports them).
enum : int { kStatusTimeoutBit = 1, kStatusCapacityBit = 2, kStatusBadPageBit = 4 };

// Per-device lookups of zyfa_api.cu (cached per device): the status word's address, the SM count.
// nullptr / 0 if the CUDA call behind them fails.
int* device_status_word(int dev);
int device_sm_count(int dev);

// cuTensorMapEncodeTiled with unit element strides' usual options; false if the driver refuses the map.
bool encode_tensor_map(CUtensorMap* m, CUtensorMapDataType type, unsigned rank, void* base, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t* estr, CUtensorMapSwizzle sw);

// Strides in bytes; an offset is formed in 64 bits, since a long cache passes 2^31 bytes and elements.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  long long num_pages;
  long long k_page, k_tok, k_head, v_page, v_tok, v_head;
  int page_size, H_kv;
};

// Of the scales of a 4-bit cache, in bytes.
struct ScaleView {
  uint8_t* k;
  uint8_t* v;
  long long k_page, k_tok, k_head, v_page, v_tok, v_head;
};

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// `rows` runs of `bytes` bytes, `stride` bytes apart (none for a null pointer).
struct Span {
  uintptr_t begin, end;
  long long bytes, rows, stride;
  Span(const void* p, long long bytes_, long long rows_ = 1, long long stride_ = 0) : bytes(bytes_), rows(rows_), stride(stride_) {
    const bool any = p && bytes > 0 && rows > 0;
    begin = any ? reinterpret_cast<uintptr_t>(p) : 0;
    end = any ? begin + static_cast<uintptr_t>(rows - 1) * static_cast<uintptr_t>(stride) + static_cast<uintptr_t>(bytes) : 0;
  }
};

// A dense output and `x` have a byte in common.
inline bool overlap(const Span& out, const Span& x) {
  if (out.end <= x.begin || x.end <= out.begin) return false;
  if (x.rows == 1 || out.begin < x.begin + x.bytes) return true;
  if (x.stride <= 0) return false;
  const uintptr_t i = (out.begin - x.begin - x.bytes) / x.stride + 1;  // the first run that ends behind out's beginning
  return x.begin + i * x.stride < out.end;
}

// Of what strides count: values, or bytes of two e2m1 codes.
inline int element_size(zyfa_dtype_t t) { return t == ZYFA_DTYPE_BF16 ? 2 : 1; }
inline long long row_bytes(zyfa_dtype_t t, int D) { return t == ZYFA_DTYPE_E2M1 ? D / 2 : static_cast<long long>(D) * element_size(t); }

enum : unsigned { kWideCaches = 1u << ZYFA_DTYPE_E4M3 | 1u << ZYFA_DTYPE_BF16, k4BitCaches = 1u << ZYFA_DTYPE_E2M1 };

inline zyfa_status_t check_cache(const zyfa_paged_cache_t* c, CacheView* view, unsigned types = kWideCaches) {
  if (!c) return ZYFA_ERR_INVALID_ARG;
  if (static_cast<unsigned>(c->dtype) > 2u || !((types >> c->dtype) & 1)) return ZYFA_ERR_INVALID_ARG;
  if (c->page_size < 1 || c->page_size > 65536 || c->num_pages < 1 || c->H_kv < 1) return ZYFA_ERR_INVALID_ARG;
  const bool shape_ok = (c->D_qk == 64 && c->D_v == 64) || (c->D_qk == 128 && c->D_v == 128) ||
                        (c->D_qk == 192 && c->D_v == 128);
  if (!shape_ok) return ZYFA_ERR_UNSUPPORTED;
  if (!c->k || !c->v) return ZYFA_ERR_INVALID_ARG;
  const long long es = element_size(c->dtype);
  const long long strides[6] = {c->k_page_stride, c->k_token_stride, c->k_head_stride,
                                c->v_page_stride, c->v_token_stride, c->v_head_stride};
  bool whole = aligned(c->k, 16) && aligned(c->v, 16);
  for (long long s : strides) {
    if (s < 0) return ZYFA_ERR_INVALID_ARG;
    if (s > (1ll << 46)) return ZYFA_ERR_UNSUPPORTED;
    whole = whole && (s * es) % 16 == 0;
  }
  if (!whole) return ZYFA_ERR_MISALIGNED;
  if (c->num_pages > (1ll << 31) - 1) return ZYFA_ERR_UNSUPPORTED;  // page numbers are int32
  view->k = static_cast<uint8_t*>(c->k);
  view->v = static_cast<uint8_t*>(c->v);
  view->num_pages = c->num_pages;
  view->k_page = c->k_page_stride * es;
  view->k_tok = c->k_token_stride * es;
  view->k_head = c->k_head_stride * es;
  view->v_page = c->v_page_stride * es;
  view->v_tok = c->v_token_stride * es;
  view->v_head = c->v_head_stride * es;
  view->page_size = c->page_size;
  view->H_kv = c->H_kv;
  return ZYFA_OK;
}

inline zyfa_status_t check_scales(const zyfa_paged_scales_t* s, ScaleView* view) {
  if (!s || !s->k || !s->v) return ZYFA_ERR_INVALID_ARG;
  bool whole = aligned(s->k, 4) && aligned(s->v, 4);
  for (long long x : {s->k_page_stride, s->k_token_stride, s->k_head_stride, s->v_page_stride, s->v_token_stride, s->v_head_stride}) {
    if (x < 0) return ZYFA_ERR_INVALID_ARG;
    if (x > (1ll << 46)) return ZYFA_ERR_UNSUPPORTED;
    whole = whole && x % 4 == 0;
  }
  if (!whole) return ZYFA_ERR_MISALIGNED;
  *view = {static_cast<uint8_t*>(s->k), static_cast<uint8_t*>(s->v), s->k_page_stride, s->k_token_stride, s->k_head_stride,
           s->v_page_stride, s->v_token_stride, s->v_head_stride};
  return ZYFA_OK;
}

// floor(t / size) = t * magic >> shift for t < 2^bits (bits at most 31) and size of 1 to 65536: with s = ceil(log2 size) and
// magic = floor(2^(bits + s) / size) + 1 the error of t * magic / 2^(bits + s) is below 1 / size.
inline void division_by(int size, int bits, uint32_t* magic, int* shift) {
  int s = 0;
  while ((1 << s) < size) ++s;
  *shift = bits + s;
  *magic = static_cast<uint32_t>((1ull << (bits + s)) / static_cast<unsigned>(size) + 1);
}

// Programmatic dependent launch: the kernel may start while its predecessor on the stream still runs, and waits for it
// on the device (wait_for_predecessor, before it touches memory), so that its launch costs the stream nothing.  Its inputs
// are written within its lifetime, so it reads them by ordinary loads, which the wait orders, not as read-only data.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned block, int smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The two e2m1 codes of byte I of `x`, the lower one first, as fp16 (exact).
template <int I>
__device__ __forceinline__ uint32_t widen_e2m1(uint32_t x) {
  uint32_t d;
  if constexpr (I == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(d) : "r"(x));
  else if constexpr (I == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(d) : "r"(x));
  else if constexpr (I == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(d) : "r"(x));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(d) : "r"(x));
  return d;
}
// Two e4m3 codes (low half of `x`) as fp16 (exact).
__device__ __forceinline__ uint32_t widen_e4m3(uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t widen_e4m3_hi(uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(x));
  return d;
}
// An e2m1 code times an e4m3 scale has 6 bits and lies between 2^-10 and 2688: exact in fp16.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two products by one instruction.
__device__ __forceinline__ float2 times(float a, float b, float f) {
  float2 d;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a), "f"(b), "f"(f));
  return d;
}

__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// A load that sees what had been written when it was issued (from L2, not from an earlier copy in this SM's L1).
__device__ __forceinline__ int load_relaxed(const int* p) {
  int x;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace zyfa
