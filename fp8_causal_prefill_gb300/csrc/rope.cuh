// What the kernels that rotate and store share: angles of far positions, the rotation of channel pairs, a block's walk over its tokens'
// heads, and the host's checks of a rotation and of caches that are written.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <utility>

#include "paged.cuh"

namespace zyfa {
namespace rope {

constexpr int kMaxTokens = 32;  // tokens per block at most

// A multiple of the 16-channel pieces of a key head and of a value head.
template <int DQK>
constexpr int kThreads = DQK == 192 ? 192 : 256;

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

// The page of a slot, not below 0, and the token's place in it.
__device__ __forceinline__ void place_of(long long slot, int page_size, long long* page, long long* off) {
  if (slot <= 0x7fffffffll) {
    *page = static_cast<unsigned>(slot) / static_cast<unsigned>(page_size);
    *off = static_cast<unsigned>(slot) % static_cast<unsigned>(page_size);
  } else {
    *page = slot / page_size;
    *off = slot % page_size;
  }
}

// Cosines and sines of the turns of tokens n0 to n0 + here - 1, by a block of THREADS: a thread keeps its pair, THREADS / half
// tokens at a time.
template <int THREADS, int HALF, typename Args>
__device__ __forceinline__ void fill_turns(const Args& a, long long n0, int here, float (&s_cos)[kMaxTokens][HALF], float (&s_sin)[kMaxTokens][HALF]) {
  const int tid = threadIdx.x, half = a.rot / 2;
  if (half > 0) {
    const int at_once = THREADS / half, t0 = tid / half, p = tid - t0 * half;
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
}

__device__ __forceinline__ float inverse(const float* desc, int i) { return desc ? __frcp_rn(desc[i]) : 1.0f; }

__device__ __forceinline__ void widen8(const uint4& x, float (&y)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = __uint_as_float(w[i] << 16);
    y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
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

// A rotation's checks; fills in the arguments' rot, offset, axis_end and inv_freq (left as they are without one).
template <typename Args>
zyfa_status_t set_rope(Args& a, const zyfa_rope_t* rope, int D_qk, long long N, const int* positions, long long position_stride) {
  if (!rope || rope->rot_dim == 0) return ZYFA_OK;
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
  return ZYFA_OK;
}

}  // namespace rope
}  // namespace zyfa
