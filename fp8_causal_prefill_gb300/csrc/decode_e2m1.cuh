// Attention of one new token per request over a 4-bit paged cache: device code.
//
// The mathematics, the split of the work over requests, its schedule and the join are those of the e4m3 and bf16 caches
// (decode.cuh): one pass with the running maximum and sum, tiles of all requests numbered one after the other and dealt evenly, parts
// joined in order.  What differs is a tile: codes and scales come in, and are widened where they are used.
//
// * Products run with keys (or channels of V) as the rows of mma.sync.m16n8k16 and query heads as its 8 columns, in fp16: a code
//   times its scale has 6 bits and is exact there, and a bf16 query is, over a power of two near its row's largest.
// * K: the contraction may take the channels in any order, so lane 4g + t keeps 32 neighbouring channels of key g (16 bytes: one
//   wide read of shared memory, conversions two values at a time in place, two scales) and the same channels of the queries.
// * V: the contraction runs over keys, two of which share a register, while the two codes of a byte are channels.  ldmatrix
//   transposes 16-bit elements, four channels of a key, so that a register holds them for two keys; each byte is converted and
//   halves of pairs exchanged: 3 operations for 2 values, with the scale's product.
// * Codes are numbers whatever their bits, so what lies in shared memory behind a request's end only needs scales of 0.
//
// Bound: HBM, 9/16 byte a value, and next to it the ALU that converts: a key and head of 128 channels takes some 8 of its
// warp instructions for 144 bytes.
#pragma once
#include "decode.cuh"

namespace zyfa {
namespace decode4 {

using namespace decode;

constexpr int kKeys = 32;         // of a warp's turn
constexpr int kWarps = 4;         // compute warps of a block at most
constexpr int kStages = 3;        // of the ring at most
constexpr int kMaxTokens = kWarps * kKeys;

struct Args : DecodeArgs {
  ScaleView scales;
  int boxes;             // codes and scales come by TMA, box by box (1 << box_log2 tokens of a page); else piece by piece, and box_log2 is the tile's
  int dense;             // the scales of a box are one run of bytes
  int k_log2, v_log2;    // tokens whose rows share 128 bytes of shared memory (log2), where a block's heads take less
  int k_unit, v_unit;    // bytes of scales copied at a time: 4, 8, or 16 across heads
  uint32_t order;        // the key within 8 that row g of the scores is: nibble g
};

struct Maps4 {
  CUtensorMap k, v, ks, vs;
};

template <int DQK, int DV>
struct Tile4 {
  static constexpr int kRowK = DQK / 2, kRowV = DV / 2, kScaleK = DQK / 16, kScaleV = DV / 16;
  static constexpr int kKeyBytes = kRowK + kRowV + kScaleK + kScaleV;
};

// Codes of a tile lie in shared memory box by box, a token's heads one after the other, in columns of 128 bytes [token][128] with
// the 16-byte pieces of a row exchanged by its number, as TMA's 128-byte swizzle does; rows of 32 or 64 bytes share 128 (`log2`).
struct Place {
  int log2, box_log2;
  uint32_t box_bytes;
  __device__ __forceinline__ uint32_t operator()(int token, int byte) const {
    const int in = token & ((1 << box_log2) - 1), row = in >> log2, inner = ((in & ((1 << log2) - 1)) << (7 - log2)) + byte;
    return (token >> box_log2) * box_bytes + (inner >> 7) * (128u << (box_log2 - log2)) + row * 128 + ((((inner >> 4) ^ row) & 7) << 4) + (inner & 15);
  }
  // of a multiple of 16 tokens, from token 0
  __device__ __forceinline__ uint32_t step(int token) const {
    return (token >> box_log2) * box_bytes + ((token & ((1 << box_log2) - 1)) >> log2) * 128;
  }
};
__host__ __device__ inline uint32_t bytes4(int tokens, int pitch, int log2) { return static_cast<uint32_t>(tokens >> log2) * 128u * ((pitch + 127) / 128); }
inline int share_log2(int pitch) { return pitch == 32 ? 2 : pitch == 64 ? 1 : 0; }

__device__ __forceinline__ int key4(uint32_t order, int g) { return order >> (4 * g) & 7; }

// 4 or 8 bytes global -> shared; `bytes` 0 writes zeros without reading.
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
               : "memory");
}
// The barrier counts this lane once all its copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 x;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t lds2(uint32_t addr) {
  uint16_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t lds1(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// (a.lo s, b.lo s') and (a.hi s, b.hi s') from s0 = (s, 0) and s1 = (0, s'): exact, since one of the two products in each half is 0.
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b, uint32_t s0, uint32_t s1) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 x, y;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 x, {l, l};\n\tmov.b32 {l, h}, %2;\n\tmov.b32 y, {l, l};\n\t"
      "mul.rn.f16x2 y, y, %4;\n\tfma.rn.f16x2 %0, x, %3, y;\n\t}"
      : "=r"(d)
      : "r"(a), "r"(b), "r"(s0), "r"(s1));
  return d;
}
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b, uint32_t s0, uint32_t s1) {
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 x, y;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 x, {h, h};\n\tmov.b32 {l, h}, %2;\n\tmov.b32 y, {h, h};\n\t"
      "mul.rn.f16x2 y, y, %4;\n\tfma.rn.f16x2 %0, x, %3, y;\n\t}"
      : "=r"(d)
      : "r"(a), "r"(b), "r"(s0), "r"(s1));
  return d;
}
__device__ __forceinline__ void apart(uint32_t s, uint32_t (&d)[2]) {
  d[0] = s & 0xffffu;
  d[1] = s & 0xffff0000u;
}
__device__ __forceinline__ uint32_t halves(float lo, float hi) { return pack2<true>(lo, hi); }

// Where a lane reads a warp's run of 32 keys, relative to the run's first key (a multiple of 32): K of keys 8u + row, V of 16 keys.
// 16 keys on, the exchange of pieces is the same unless four tokens share a row (64 channels, one head).
template <int DQK, int DV>
struct Reader4 {
  static constexpr bool kWideK = DQK >= 128, kRestK = DQK % 128 != 0;  // 64 bytes of a row by 16, 32 by 8
  static constexpr int kPairsV = DV / 64;                              // 32-channel pieces of V, two at a time
  uint32_t wide[2], rest[kWideK ? 1 : 4], value[kPairsV == 1 ? 2 : 1][kPairsV];
  uint32_t k_16, v_16;               // from 16 keys to the next
  uint32_t k_scale, v_scale[2];      // of key g, and of keys 2t and 2t + 1 (of each 8)
  uint32_t k_scale_8, v_scale_8;     // from 8 keys to the next

  __device__ __forceinline__ void set(const Args& a, int lane, int head, int first, const Place& kp, const Place& vp) {
    using T = Tile4<DQK, DV>;
    const int g = lane >> 2, t = lane & 3;
    const int kb = head * T::kRowK, vb = head * T::kRowV;
    k_16 = kp.step(16);
    v_16 = vp.step(16);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int key = first + 8 * u + key4(a.order, g);
      if (kWideK && u < 2) wide[u] = kp(key, kb + 16 * t);
      if (kRestK && u < (kWideK ? 1 : 4)) rest[u] = kp(key, kb + (kWideK ? 64 : 0) + 8 * t);
    }
#pragma unroll
    for (int n = 0; n < (kPairsV == 1 ? 2 : 1); ++n)
#pragma unroll
      for (int p = 0; p < kPairsV; ++p)
        value[n][p] = vp(first + 16 * n + (lane >> 3 & 1) * 8 + key4(a.order, lane & 7), vb + 32 * p + (lane >> 4) * 16);
    const int ks = a.heads * T::kScaleK, vs = a.heads * T::kScaleV;
    k_scale = (first + key4(a.order, g)) * ks + head * T::kScaleK;
    v_scale[0] = (first + key4(a.order, 2 * t)) * vs + head * T::kScaleV;
    v_scale[1] = (first + key4(a.order, 2 * t + 1)) * vs + head * T::kScaleV;
    k_scale_8 = 8 * ks;
    v_scale_8 = 8 * vs;
  }
  __device__ __forceinline__ uint32_t wide_at(int u) const { return wide[u & 1] + (u >> 1) * k_16; }
  // (192 channels: rows of 96 bytes share nothing, and 8 keys on is 1 KiB)
  __device__ __forceinline__ uint32_t rest_at(int u) const { return kWideK ? rest[0] + (u & 1) * 1024 + (u >> 1) * k_16 : rest[kWideK ? 0 : u]; }
  __device__ __forceinline__ uint32_t value_at(int n, int p) const { return kPairsV == 1 ? value[kPairsV == 1 ? n : 0][p] : value[0][p] + n * v_16; }
};

// Where a run's first key lies in a stage's K, V and their scales.
struct Run4 {
  uint32_t k, v, ks, vs;
};

// A lane's share of a tile's scales, [token][head] in shared memory: `unit` bytes at a time, the pieces of a token's heads one after the other.
struct ScaleCopy {
  int unit, first, piece, step, rest, all, each, pitch;
  const uint8_t* from;
  long long head_stride, offset;
  __device__ __forceinline__ ScaleCopy(int unit_, int heads, int heads_apart, int bytes, const uint8_t* from_, long long head_stride_, int lane)
      : unit(unit_), pitch(heads_apart * bytes), from(from_), head_stride(head_stride_) {
    all = heads * bytes / unit;
    each = unit == 16 ? all : bytes / unit;  // 16 bytes only where heads follow one another
    first = lane / all;
    piece = lane - first * all;
    step = 32 / all;
    rest = 32 - step * all;
    offset = at(piece);
  }
  __device__ __forceinline__ long long at(int p) const { return p / each * head_stride + p % each * unit; }
  template <int UNIT>
  __device__ __forceinline__ void copy_by(const long long* rows, int tokens, uint32_t to) const {
    int r = first, p = piece;
    long long off = offset;
    while (r < tokens) {
      const long long row = rows[r];
      const uint8_t* src = from + off + (row < 0 ? 0 : row);
      const uint32_t dst = to + r * pitch + p * UNIT;
      if constexpr (UNIT == 16)
        copy16(dst, src, row < 0 ? 0 : 16);
      else
        copy_small<UNIT>(dst, src, row < 0 ? 0 : UNIT);
      r += step;
      if (rest) {
        p += rest;
        if (p >= all) {
          p -= all;
          ++r;
        }
        off = at(p);
      }
    }
  }
  __device__ __forceinline__ void copy(const long long* rows, int tokens, uint32_t to) const {
    if (unit == 16)
      copy_by<16>(rows, tokens, to);
    else if (unit == 8)
      copy_by<8>(rows, tokens, to);
    else
      copy_by<4>(rows, tokens, to);
  }
};

// ------------------------------------------------------------------------------------------------
// the state of a compute warp: up to 8 NC query heads against its tiles

template <int DQK, int DV, int NC>
struct Rows4 {
  using T = Tile4<DQK, DV>;
  using R = Reader4<DQK, DV>;
  static constexpr int KB = kKeys / 16, kKSteps = DQK / 16, kPieces = DV / 32;
  static constexpr float kLift = 15.0f;             // weights in fp16 up to 2^15, so that light ones keep their bits
  static constexpr float kNoKey = 3.402823466e38f;  // ref before the first key: lifts every score above its negative over the limit

  uint32_t qf[NC][kKSteps][2];  // B fragments of the queries
  float o[NC][kPieces][2][4], m[NC][2], l[NC][2];  // this lane's two heads of each 8
  F2 ref[NC], scale[NC];
  float dv;

  // A query's 16 neighbouring channels as B fragments; they are bits of two bf16 values a word.
  static __device__ __forceinline__ uint32_t top_bits(uint32_t top, uint32_t w) { return max(top, max(w & 0x7fff0000u, (w << 16) & 0x7fff0000u)); }

  // Begins a request's part: its queries from shared memory, `count` dense bf16 rows.
  __device__ __forceinline__ void begin(uint32_t queries, int count, float scale_, float dv_, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      // rows behind the last head repeat it: their columns are computed and never written
      const uint32_t row = queries + min(8 * c + (lane >> 2), count - 1) * (DQK * 2);
      uint32_t w[DQK / 8];  // this lane's channels, two a word
      if constexpr (R::kWideK) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = lds16(row + 64 * t + 16 * i);
          w[4 * i] = x.x;
          w[4 * i + 1] = x.y;
          w[4 * i + 2] = x.z;
          w[4 * i + 3] = x.w;
        }
      }
      if constexpr (R::kRestK) {
        constexpr int at = R::kWideK ? 16 : 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 x = lds16(row + (R::kWideK ? 256 : 0) + 32 * t + 16 * i);
          w[at + 4 * i] = x.x;
          w[at + 4 * i + 1] = x.y;
          w[at + 4 * i + 2] = x.z;
          w[at + 4 * i + 3] = x.w;
        }
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < DQK / 8; ++i) top = top_bits(top, w[i]);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest magnitude to [2^14, 2^15), which an infinity or NaN stays beyond
      const int shift = min(127, 141 - static_cast<int>(top >> 23));
      const float f = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
      for (int i = 0; i < kKSteps; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t x = w[2 * i + j];
          qf[c][i][j] = halves(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
        }
      const float undo = ldexpf(scale_, -shift);
      scale[c] = {__shfl_sync(0xffffffffu, undo, 8 * t), __shfl_sync(0xffffffffu, undo, 8 * t + 4)};
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) o[c][i][j][0] = o[c][i][j][1] = o[c][i][j][2] = o[c][i][j][3] = 0.0f;
      m[c][0] = m[c][1] = -INFINITY;
      ref[c] = {kNoKey, kNoKey};
      l[c][0] = l[c][1] = 0.0f;
    }
    dv = dv_;
  }

  // Two steps of the contraction: a word of key g and one of key g + 8, of one scale each.
  __device__ __forceinline__ void two_steps(float (&x)[NC][4], int step, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb) {
    const uint32_t a0 = mul_f16x2(widen_e2m1<0>(a), sa), a1 = mul_f16x2(widen_e2m1<0>(b), sb);
    const uint32_t a2 = mul_f16x2(widen_e2m1<1>(a), sa), a3 = mul_f16x2(widen_e2m1<1>(b), sb);
#pragma unroll
    for (int c = 0; c < NC; ++c) mma<kF16>(x[c], a0, a1, a2, a3, qf[c][step][0], qf[c][step][1]);
    const uint32_t b0 = mul_f16x2(widen_e2m1<2>(a), sa), b1 = mul_f16x2(widen_e2m1<2>(b), sb);
    const uint32_t b2 = mul_f16x2(widen_e2m1<3>(a), sa), b3 = mul_f16x2(widen_e2m1<3>(b), sb);
#pragma unroll
    for (int c = 0; c < NC; ++c) mma<kF16>(x[c], b0, b1, b2, b3, qf[c][step + 1][0], qf[c][step + 1][1]);
  }

  // One run of 32 keys.  mask: those that count.
  __device__ __forceinline__ void tile(const Run4& s, const R& at, uint32_t order, uint32_t mask, int lane) {
    const int g = lane >> 2, t = lane & 3;
    // S^T: rows are keys, columns heads; then scores in units of log2
    F2 x[NC][KB][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float acc[NC][4];
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c][0] = acc[c][1] = acc[c][2] = acc[c][3] = 0.0f;
      const uint32_t scales = s.ks + at.k_scale + 2 * kb * at.k_scale_8, scales_8 = scales + at.k_scale_8;
      if constexpr (R::kWideK) {
        const uint4 ka = lds16(s.k + at.wide_at(2 * kb)), kc = lds16(s.k + at.wide_at(2 * kb + 1));
        // the scales of this lane's two blocks of channels, of both keys
        const uint32_t sa = widen_e4m3(lds2(scales + 2 * t)), sc = widen_e4m3(lds2(scales_8 + 2 * t));
        const uint32_t sa0 = prmt(sa, sa, 0x1010), sa1 = prmt(sa, sa, 0x3232), sc0 = prmt(sc, sc, 0x1010), sc1 = prmt(sc, sc, 0x3232);
        two_steps(acc, 0, ka.x, kc.x, sa0, sc0);
        two_steps(acc, 2, ka.y, kc.y, sa0, sc0);
        two_steps(acc, 4, ka.z, kc.z, sa1, sc1);
        two_steps(acc, 6, ka.w, kc.w, sa1, sc1);
      }
      if constexpr (R::kRestK) {
        constexpr int first = R::kWideK ? 8 : 0;
        const uint2 ka = lds8(s.k + at.rest_at(2 * kb)), kc = lds8(s.k + at.rest_at(2 * kb + 1));
        const uint32_t sa = widen_e4m3(lds1(scales + first + t) * 0x101u), sc = widen_e4m3(lds1(scales_8 + first + t) * 0x101u);
        two_steps(acc, first, ka.x, kc.x, sa, sc);
        two_steps(acc, first + 2, ka.y, kc.y, sa, sc);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c][kb][0] = mul2({acc[c][0], acc[c][1]}, scale[c]);
        x[c][kb][1] = mul2({acc[c][2], acc[c][3]}, scale[c]);
      }
    }
    if (mask != 0xffffffffu) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (!((mask >> (kb * 16 + j * 8 + key4(order, g))) & 1))
#pragma unroll
            for (int c = 0; c < NC; ++c) x[c][kb][j] = {-INFINITY, -INFINITY};
    }
    uint32_t pf[NC][KB][2];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      // The reference m moves only when a key exceeds it: log2 of a weight is then above the lift.
      F2 y[KB][2];
      float over = -INFINITY;
      auto weigh = [&]() {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y[kb][j] = add2(x[c][kb][j], ref[c]);
            over = fmaxf(over, fmaxf(y[kb][j].x, y[kb][j].y));
          }
      };
      weigh();
      if (__any_sync(0xffffffffu, over > kLift)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = m[c][e];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
            top = e ? fmaxf(top, fmaxf(x[c][kb][0].y, x[c][kb][1].y)) : fmaxf(top, fmaxf(x[c][kb][0].x, x[c][kb][1].x));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const bool none = top == -INFINITY;
          const float f = none ? 1.0f : exp2_approx(m[c][e] - top);
          m[c][e] = top;
          (e ? ref[c].y : ref[c].x) = none ? kNoKey : kLift - top;
          l[c][e] *= f;
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              o[c][i][j][e] *= f;
              o[c][i][j][e + 2] *= f;
            }
        }
        weigh();
      }
      // weights, transposed into the B operand (keys are now the contraction)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const F2 w = {exp2_approx(y[kb][j].x), exp2_approx(y[kb][j].y)};
          const F2 sum = add2({l[c][0], l[c][1]}, w);
          l[c][0] = sum.x;
          l[c][1] = sum.y;
          pf[c][kb][j] = transpose8x8(halves(w.x, w.y));
        }
    }
    // O^T += V^T P^T: rows are channels of V, the contraction keys 2t, 2t + 1 of each 8 (in the scores' order)
    const uint32_t pick = g < 4 ? 0x6240u : 0x7351u;  // of two keys' scales: those of this lane's block of every 32 channels
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t sv[2][kPieces][2];  // scales of keys 2t, 2t + 1 of the first 8 and of the second: (s, 0) and (0, s)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t base = s.vs + (2 * kb + j) * at.v_scale_8, first = base + at.v_scale[0], second = base + at.v_scale[1];
        if constexpr (DV == 128) {
          const uint2 a = lds8(first), b = lds8(second);
          const uint32_t lo = prmt(a.x, b.x, pick), hi = prmt(a.y, b.y, pick);
          apart(widen_e4m3(lo), sv[j][0]);
          apart(widen_e4m3_hi(lo), sv[j][1]);
          apart(widen_e4m3(hi), sv[j][2]);
          apart(widen_e4m3_hi(hi), sv[j][3]);
        } else {
          const uint32_t lo = prmt(lds4(first), lds4(second), pick);
          apart(widen_e4m3(lo), sv[j][0]);
          apart(widen_e4m3_hi(lo), sv[j][1]);
        }
      }
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        uint32_t r[4];
        if (p % 2 == 0) {
          ldsm4t(s.v + at.value_at(kb, p / 2), r);
          two_pieces[0] = r[2];
          two_pieces[1] = r[3];
        } else {
          r[0] = two_pieces[0];
          r[1] = two_pieces[1];
        }
        uint32_t f[2][4];  // [8 keys][channel]: keys 2t and 2t + 1
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t c0 = widen_e2m1<0>(r[j]), c1 = widen_e2m1<1>(r[j]), c2 = widen_e2m1<2>(r[j]), c3 = widen_e2m1<3>(r[j]);
          f[j][0] = pair_lo(c0, c2, sv[j][p][0], sv[j][p][1]);
          f[j][1] = pair_hi(c0, c2, sv[j][p][0], sv[j][p][1]);
          f[j][2] = pair_lo(c1, c3, sv[j][p][0], sv[j][p][1]);
          f[j][3] = pair_hi(c1, c3, sv[j][p][0], sv[j][p][1]);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          mma<kF16>(o[c][p][0], f[0][0], f[0][1], f[1][0], f[1][1], pf[c][kb][0], pf[c][kb][1]);
          mma<kF16>(o[c][p][1], f[0][2], f[0][3], f[1][2], f[1][3], pf[c][kb][0], pf[c][kb][1]);
        }
      }
    }
  }

  // Ends a request's part: writes its rows (`count` query heads from `first`), or (m, l, O) to part `slot` of the workspace.
  __device__ __forceinline__ void finish(const DecodeArgs& a, int b, int first, int count, bool direct, long long slot, int lane) {
    const int g = lane >> 2;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sum = total(c, e);
        const int head = 8 * c + (lane & 3) * 2 + e;
        if (head < count) {
          const long long row = (direct ? static_cast<long long>(b) : slot) * a.H + first + head;
          const float f = !direct ? dv : sum == 0.0f ? 0.0f : dv / sum;
          if (g == 0) put_sums(a, row, direct, m[c][e], sum);
          if (direct) {
            __nv_bfloat16* out = a.out + row * DV + 4 * g;
#pragma unroll
            for (int p = 0; p < kPieces; ++p)
              *reinterpret_cast<uint2*>(out + 32 * p) = make_uint2(pack2<false>(o[c][p][0][e] * f, o[c][p][0][e + 2] * f),
                                                                   pack2<false>(o[c][p][1][e] * f, o[c][p][1][e + 2] * f));
          } else {
            put_o(a.part + row * DV, c, e, f, g);
          }
        }
      }
  }

  // The same for a request's part whose tiles' token runs `subs` warps shared (this one the sub-th): they leave (m, l, O) in
  // shared memory, meet, join them in order, each warp some of the heads, and meet again before the memory is used anew.
  // all_ml, all_o: [subs][8 NC] and [subs][8 NC][DV], `stride` warps from one sub's to the next; meet() is false if it gave up.
  template <typename F>
  __device__ __forceinline__ bool finish_shared(const DecodeArgs& a, int b, int first, int count, bool direct, long long slot, int lane, int sub,
                                                int subs, int stride, float2* all_ml, float* all_o, F meet) {
    constexpr int kHeads = 8 * NC;
    const int g = lane >> 2;
    float2* my_ml = all_ml + sub * stride * kHeads;
    float* my_o = all_o + sub * stride * kHeads * DV;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float sum = total(c, e);
        const int head = 8 * c + (lane & 3) * 2 + e;
        if (g == 0) my_ml[head] = make_float2(m[c][e], sum);
        put_o(my_o + head * DV, c, e, dv, g);
      }
    if (!meet()) return false;
    constexpr int V = DV / 32;
    for (int head = sub; head < count; head += subs) {
      float M = -INFINITY, L = 0.0f, x[V] = {};
      for (int k = 0; k < subs; ++k) M = fmaxf(M, all_ml[k * stride * kHeads + head].x);
      for (int k = 0; k < subs; ++k) {
        const float2 ml = all_ml[k * stride * kHeads + head];
        const float e = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - M);  // 0 for a run without a valid key, whose O is 0
        L = fmaf(ml.y, e, L);
        const float* y = all_o + (k * stride * kHeads + head) * DV + lane * V;
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = fmaf(y[j], e, x[j]);
      }
      const long long row = (direct ? static_cast<long long>(b) : slot) * a.H + first + head;
      if (lane == 0) put_sums(a, row, direct, M, L);
      const float f = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
      for (int j = 0; j < V; j += 2) {
        if (direct)
          *reinterpret_cast<__nv_bfloat162*>(a.out + row * DV + lane * V + j) = __floats2bfloat162_rn(x[j] * f, x[j + 1] * f);
        else
          *reinterpret_cast<float2*>(a.part + row * DV + lane * V + j) = make_float2(x[j], x[j + 1]);
      }
    }
    return meet();
  }

 private:
  uint32_t two_pieces[2];  // the second piece of a pair that one ldmatrix read

  __device__ __forceinline__ float total(int c, int e) const {
    float sum = l[c][e];
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    return sum;
  }
  static __device__ __forceinline__ void put_sums(const DecodeArgs& a, long long row, bool direct, float top, float sum) {
    if (!direct)
      a.ml[row] = make_float2(top - kLift, sum);
    else if (a.lse)
      a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum) - kLift) * 0.69314718055994531f;
  }
  // channels 4g to 4g + 3 of each 32
  __device__ __forceinline__ void put_o(float* to, int c, int e, float f, int g) const {
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      *reinterpret_cast<float4*>(to + 32 * p + 4 * g) = make_float4(o[c][p][0][e] * f, o[c][p][0][e + 2] * f, o[c][p][1][e] * f, o[c][p][1][e + 2] * f);
  }
};

// ------------------------------------------------------------------------------------------------

template <int DQK, int DV, int NC>
__global__ void __launch_bounds__((kWarps + 1) * 32, NC == 1 ? 3 : 2) decode4_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps4 maps) {
  using T = Tile4<DQK, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ unsigned s_prefix[(kWarps + 1) * 32], s_sums[kWarps + 1];
  __shared__ __align__(16) Header s_header[kStages];
  __shared__ float2 s_scale[kStages][kWarps];  // of the scores, and of V
  __shared__ long long s_row[4][kMaxTokens];   // where a tile's tokens lie in the scales of K and V, and (no boxes) in K and V; below 0: nowhere
  __shared__ unsigned s_mask[kStages][kWarps]; // its keys that count, 32 a word
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_meet[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x >> 5) - 1;  // compute warps; the next one loads
  const int S = a.stages, TT = a.tile_tokens, k_pitch = a.heads * T::kRowK, v_pitch = a.heads * T::kRowV;
  // a stage: K, V, scales of K, scales of V, queries
  const uint32_t k_bytes = bytes4(TT, k_pitch, a.k_log2), v_bytes = bytes4(TT, v_pitch, a.v_log2);
  const uint32_t ks_at = k_bytes + v_bytes, vs_at = ks_at + a.heads * TT * T::kScaleK, q_at = vs_at + a.heads * TT * T::kScaleV;
  const uint32_t stage_bytes = (q_at + a.q_bytes + 1023) & ~1023u;
  const Place k_place = {a.k_log2, a.box_log2, bytes4(1 << a.box_log2, k_pitch, a.k_log2)};
  const Place v_place = {a.v_log2, a.box_log2, bytes4(1 << a.box_log2, v_pitch, a.v_log2)};
  const uint32_t tiles_s = smem_addr(smem), full_s = smem_addr(s_full), empty_s = smem_addr(s_empty);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full_s + 8 * i, a.boxes ? 1 : 33);  // the header, and (piece by piece) each lane's copies
      ptx::mbar_init(empty_s + 8 * i, warps);
    }
    for (int i = 0; i < a.heads * a.chunk_warps; ++i) ptx::mbar_init(smem_addr(s_meet + i), a.subs);
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (a.boxes && threadIdx.x == 32) {
    ptx::tma_prefetch_desc(&maps.k);
    ptx::tma_prefetch_desc(&maps.v);
    if (!a.dense) {
      ptx::tma_prefetch_desc(&maps.ks);
      ptx::tma_prefetch_desc(&maps.vs);
    }
  }
  __syncthreads();
  wait_for_predecessor();
  if (!a.whole) let_successor_start();  // to the join

  // this block: group g, KV heads from head0, chunks of query heads from chunk0
  const unsigned g = blockIdx.x / a.units;
  const int unit = blockIdx.x % a.units, chunk_units = (a.chunks + a.chunk_warps - 1) / a.chunk_warps;
  const int head0 = unit / chunk_units * a.heads, chunk0 = unit % chunk_units * a.chunk_warps;
  Schedule plan;
  int b, left;
  unsigned tile0;
  if (a.whole) {
    b = static_cast<int>(g);
    tile0 = 0;
    left = static_cast<int>(Schedule::tiles(a, b));
  } else {
    plan.find(a, s_prefix, s_sums, true, g, &b, &tile0, &left);
  }
  // a compute warp: a run of keys, a KV head, a chunk of its query heads
  const int head = warp % a.heads, chunk = chunk0 + warp / a.heads % a.chunk_warps, sub = warp / (a.heads * a.chunk_warps);
  const int hk = head0 + head, q0 = hk * a.group + chunk * a.chunk_heads, nq = min(a.chunk_heads, a.group - chunk * a.chunk_heads);
  const bool idle = hk >= a.cache.H_kv || nq <= 0;  // the last block of a group may have heads or chunks too many
  if (left == 0) {
    if (a.whole && sub == 0 && !idle) {  // a request without tokens (the warp that loads has a larger sub)
      const long long row = static_cast<long long>(b) * a.H + q0;
      for (int i = lane; i < nq * DV / 2; i += 32) reinterpret_cast<__nv_bfloat162*>(a.out + row * DV)[i] = __floats2bfloat162_rn(0.0f, 0.0f);
      if (a.lse)
        for (int i = lane; i < nq; i += 32) a.lse[row + i] = -INFINITY;
    }
    return;
  }

  if (warp == warps) {
    if (a.stalled) return;
    const int heads = min(a.heads, a.cache.H_kv - head0);
    Cursor c;
    c.start(a, b, tile0, left);
    // the block's query rows: whole heads, or (more chunks than warps) part of one head's
    const int first_q = head0 * a.group + chunk0 * a.chunk_heads;
    const int queries = chunk_units > 1 ? min(a.chunk_warps * a.chunk_heads, a.group - chunk0 * a.chunk_heads) : heads * a.group;
    const uint8_t *k = a.cache.k + head0 * a.cache.k_head, *v = a.cache.v + head0 * a.cache.v_head;
    const uint8_t *ks = a.scales.k + head0 * a.scales.k_head, *vs = a.scales.v + head0 * a.scales.v_head;
    bool bad = false;
    int stage = 0;
    uint32_t parity = 1;  // a new barrier counts as one whose phase before its first has ended
    auto descales = [&](int st) {  // of a request that begins with this tile
      if (c.first && lane < heads) {
        const int i = a.desc_per_head ? c.b * a.desc_request + head0 + lane : 0;
        s_scale[st][lane] = {a.scale_log2 * (a.k_desc ? a.k_desc[i] : 1.0f), a.v_desc ? a.v_desc[i] : 1.0f};
      }
    };
    // What the compute warps need to know of a tile, and its queries; `bytes` of other copies count on the barrier.
    auto publish = [&](int st, uint32_t base, uint32_t bar, int valid, bool whole, uint32_t bytes) {
      s_header[st] = {c.b, c.flags(TT) | (whole ? 0 : kPartial), valid, 0};
      if (c.first) {
        bytes += queries * (DQK * 2);
        bulk_load(base + q_at, a.q + c.b * a.q_batch + static_cast<long long>(first_q) * (DQK * 2), queries * (DQK * 2), bar);
      }
      ptx::mbar_arrive_expect_tx(bar, bytes);
    };
    if (a.boxes) {
      // a lane: a box of the tile
      const int boxes = TT >> a.box_log2, row = lane << a.box_log2;
      const uint32_t ks_bytes = a.heads * T::kScaleK << a.box_log2, vs_bytes = a.heads * T::kScaleV << a.box_log2;
      const uint32_t k_to = lane * k_place.box_bytes, v_to = k_bytes + lane * v_place.box_bytes, ks_to = ks_at + lane * ks_bytes, vs_to = vs_at + lane * vs_bytes;
      const uint32_t box_bytes = k_place.box_bytes + v_place.box_bytes + ks_bytes + vs_bytes;
      const int k_column = a.k_log2 ? 0 : head0 * T::kRowK / 128, v_column = a.v_log2 ? 0 : head0 * T::kRowV / 128;
      int pg, off;
      auto look_up = [&]() {
        pg = -1;
        off = 0;
        if (lane < boxes && c.t + row < c.len) {
          int p;
          page_of(a, c.t + row, &p, &off);
          pg = a.table[c.b * a.table_stride + p];
        }
      };
      look_up();
      while (true) {
        if (!mbar_wait_bounded(empty_s + 8 * stage, parity, a.wait_clocks)) {
          if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
          break;
        }
        const uint32_t base = tiles_s + stage * stage_bytes, bar = full_s + 8 * stage;
        const int valid = min(TT, c.len - c.t);
        const bool inside = lane < boxes && row < valid, ok = inside && pg >= 0 && pg < a.cache.num_pages;
        bad |= inside && !ok;
        const unsigned there = __ballot_sync(0xffffffffu, ok);
        if (ok) {  // (the barrier's phase cannot end before the arrival below)
          tma_load_5d(base + k_to, &maps.k, bar, 0, off >> a.k_log2, k_column, 0, pg);
          tma_load_5d(base + v_to, &maps.v, bar, 0, off >> a.v_log2, v_column, 0, pg);
          if (a.dense) {
            bulk_load(base + ks_to, ks + pg * a.scales.k_page + off * a.scales.k_tok, ks_bytes, bar);
            bulk_load(base + vs_to, vs + pg * a.scales.v_page + off * a.scales.v_tok, vs_bytes, bar);
          } else {
            tma_load_3d(base + ks_to, &maps.ks, bar, head0 * T::kScaleK, off, pg);
            tma_load_3d(base + vs_to, &maps.vs, bar, head0 * T::kScaleV, off, pg);
          }
        }
        const bool whole = valid == TT && there == 0xffffffffu >> (32 - boxes);
        if (!whole)
          for (int i = 0; i < TT / 32; ++i) {
            const int r = 32 * i + lane;
            const unsigned mask = __ballot_sync(0xffffffffu, r < valid && (there >> (r >> a.box_log2) & 1));
            if (lane == 0) s_mask[stage][i] = mask;
          }
        descales(stage);
        __syncwarp();
        if (lane == 0) publish(stage, base, bar, valid, whole, __popc(there) * box_bytes);
        c.left = c.left_after(TT);
        if (c.left <= 0) break;
        c.advance(a, TT);
        look_up();
        if (++stage == S) {
          stage = 0;
          parity ^= 1;
        }
      }
      if (bad) atomicOr(a.status, kStatusBadPageBit);
      return;
    }
    const ScaleCopy k_scales(a.k_unit, heads, a.heads, T::kScaleK, ks, a.scales.k_head, lane), v_scales(a.v_unit, heads, a.heads, T::kScaleV, vs, a.scales.v_head, lane);
    constexpr int kSets = kMaxTokens / 32;
    int pg[kSets], off[kSets];  // page and place in it of tokens c.t + 32 i + lane
    auto look_up = [&]() {
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        const int t = c.t + 32 * i + lane;
        pg[i] = -1;
        off[i] = 0;
        if (32 * i < TT && t < c.len) {
          int p;
          page_of(a, t, &p, &off[i]);
          pg[i] = a.table[c.b * a.table_stride + p];
        }
      }
    };
    look_up();
    while (true) {
      if (!mbar_wait_bounded(empty_s + 8 * stage, parity, a.wait_clocks)) {
        if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
        break;
      }
      const uint32_t base = tiles_s + stage * stage_bytes, bar = full_s + 8 * stage;
      const int valid = min(TT, c.len - c.t);
      bool whole = valid == TT;
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        if (32 * i >= TT) break;
        const bool inside = 32 * i + lane < valid, ok = inside && pg[i] >= 0 && pg[i] < a.cache.num_pages;
        bad |= inside && !ok;
        const unsigned mask = __ballot_sync(0xffffffffu, ok);
        whole = whole && mask == 0xffffffffu;
        const long long page = pg[i], at = off[i];
        s_row[2][32 * i + lane] = ok ? page * a.cache.k_page + at * a.cache.k_tok : -1;
        s_row[3][32 * i + lane] = ok ? page * a.cache.v_page + at * a.cache.v_tok : -1;
        s_row[0][32 * i + lane] = ok ? page * a.scales.k_page + at * a.scales.k_tok : -1;
        s_row[1][32 * i + lane] = ok ? page * a.scales.v_page + at * a.scales.v_tok : -1;
        if (lane == 0) s_mask[stage][i] = mask;
      }
      __syncwarp();
      // codes: the pieces of a token's heads, 32 at a time
      auto codes = [&](auto pieces, const long long* rows, const uint8_t* from, long long head_stride, uint32_t to, const Place& place) {
        constexpr int kPieces = decltype(pieces)::value;
        const int all = heads * kPieces, step = 32 / all, rest = 32 % all;
        int r = lane / all, p = lane % all;
        while (r < valid) {
          const long long row = rows[r];
          if (row >= 0) copy16(to + place(r, p * 16), from + row + p / kPieces * head_stride + p % kPieces * 16, 16);
          r += step;
          p += rest;
          if (p >= all) {
            p -= all;
            ++r;
          }
        }
      };
      codes(std::integral_constant<int, T::kRowK / 16>(), s_row[2], k, a.cache.k_head, base, k_place);
      codes(std::integral_constant<int, T::kRowV / 16>(), s_row[3], v, a.cache.v_head, base + k_bytes, v_place);
      // scales [token][head]: zeros where there is no token
      k_scales.copy(s_row[0], TT, base + ks_at);
      v_scales.copy(s_row[1], TT, base + vs_at);
      descales(stage);
      arrive_after_copies(bar);
      __syncwarp();
      if (lane == 0) publish(stage, base, bar, valid, whole, 0);
      c.left = c.left_after(TT);
      if (c.left <= 0) break;
      c.advance(a, TT);
      look_up();
      if (++stage == S) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (bad) atomicOr(a.status, kStatusBadPageBit);
    copy_commit();
    copy_wait<0>();
    return;
  }

  Reader4<DQK, DV> reader;
  const int run_keys = a.turns * kKeys;
  reader.set(a, lane, head, sub * run_keys, k_place, v_place);
  const uint32_t my_query = q_at + (head * a.group + (chunk - chunk0) * a.chunk_heads) * (DQK * 2);
  // where warps that share a head's tokens meet
  const int peers = a.heads * a.chunk_warps, peer = warp % peers;
  uint8_t* meeting = smem + S * stage_bytes;
  float2* all_ml = reinterpret_cast<float2*>(meeting) + peer * 8 * NC;
  float* all_o = reinterpret_cast<float*>(meeting + warps * 64 * NC) + peer * 8 * NC * DV;
  const uint32_t meet_s = smem_addr(s_meet + peer);
  uint32_t meet_parity = 0;
  // Copies still in flight write to this block's shared memory: waits for them, again for a bounded time.
  auto give_up = [&](int st, uint32_t par) {
    for (int j = 1; j < S; ++j) {
      if (++st == S) {
        st = 0;
        par ^= 1;
      }
      mbar_wait_bounded(full_s + 8 * st, par, a.wait_clocks);
    }
    if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
  };
  Rows4<DQK, DV, NC> rows;
  int stage = 0;
  uint32_t parity = 0;
  while (true) {
    if (!mbar_wait_bounded(full_s + 8 * stage, parity, a.wait_clocks)) {
      give_up(stage, parity);
      return;
    }
    const Header h = s_header[stage];
    const uint32_t base = tiles_s + stage * stage_bytes;
    if (!idle) {
      if (h.flags & kFirst) rows.begin(base + my_query, nq, s_scale[stage][head].x, s_scale[stage][head].y, lane);
      for (int turn = 0; turn < a.turns; ++turn) {
        const uint32_t mask = h.flags & kPartial ? s_mask[stage][sub * a.turns + turn] : 0xffffffffu;
        if (mask == 0) continue;
        Run4 s = {base, base + k_bytes, base + ks_at, base + vs_at};
        if (turn) {
          s.k += k_place.step(turn * kKeys);
          s.v += v_place.step(turn * kKeys);
          s.ks += turn * 4 * reader.k_scale_8;
          s.vs += turn * 4 * reader.v_scale_8;
        }
        if (mask != 0xffffffffu && a.boxes) {
          // whatever the scales of keys that do not count hold is no number to multiply by 0
          const uint32_t mine = s.vs + (sub * run_keys + lane) * a.heads * T::kScaleV + head * T::kScaleV;
          if (!((mask >> lane) & 1))
#pragma unroll
            for (int i = 0; i < T::kScaleV; i += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(mine + i), "r"(0) : "memory");
          ptx::fence_proxy_async_smem();  // before a later TMA load into this stage
          __syncwarp();
        }
        rows.tile(s, reader, a.order, mask, lane);
      }
      if (h.flags & kLast) {
        const bool direct = h.flags & kDirect;
        const long long slot = static_cast<long long>(g) * 2 + (h.flags & kSlot1 ? 1 : 0);
        if (a.subs == 1) {
          rows.finish(a, h.b, q0, nq, direct, slot, lane);
        } else {
          const bool met = rows.finish_shared(a, h.b, q0, nq, direct, slot, lane, sub, a.subs, peers, all_ml, all_o, [&]() {
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(meet_s);
            const bool ok = mbar_wait_bounded(meet_s, meet_parity, a.wait_clocks);
            meet_parity ^= 1;
            return ok;
          });
          if (!met) {
            give_up(stage, parity);
            return;
          }
        }
      }
    }
    if (h.flags & kEnd) return;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(empty_s + 8 * stage);
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// host side

// A cache's codes (strides in bytes) as boxes of `box` tokens of a block's heads.
inline bool boxable(const Args& a, long long page, long long tok, long long head, int row, int log2, int box) {
  const int H_kv = a.cache.H_kv, pitch = a.heads * row;
  for (long long s : {page, tok, head})
    if (s <= 0 || s >= (1ll << 40)) return false;
  if (H_kv > 1 && head != row) return false;
  if (log2 > 0) return a.heads == H_kv && tok == pitch && box * pitch % 1024 == 0;  // tokens one after the other
  return pitch % 128 == 0 && H_kv * row % 128 == 0;
}

// The map of such boxes: [page][128-byte column][token][128], or of rows of 128 bytes that several tokens share.
inline bool make_map4(CUtensorMap* m, const uint8_t* base, const Args& a, long long page, long long tok, int row, int log2) {
  using u64 = cuuint64_t;
  using u32 = cuuint32_t;
  const CacheView& c = a.cache;
  const u64 dims[5] = {128, u64(c.page_size >> log2), u64(log2 ? 1 : c.H_kv * row / 128), 1, u64(c.num_pages)};
  const u64 strides[4] = {u64(log2 ? 128 : tok), 128, u64(log2 ? 128 : tok), u64(page)};
  const u32 box[5] = {128, u32(1) << (a.box_log2 - log2), u32(log2 ? 1 : a.heads * row / 128), 1, 1};
  const u32 estr[5] = {1, 1, 1, 1, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<uint8_t*>(base), dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The map of a box's scales: [page][token][heads].
inline bool make_scale_map(CUtensorMap* m, const uint8_t* base, const Args& a, long long page, long long tok, int bytes) {
  using u64 = cuuint64_t;
  using u32 = cuuint32_t;
  const u64 dims[3] = {u64(a.cache.H_kv) * bytes, u64(a.cache.page_size), u64(a.cache.num_pages)}, strides[2] = {u64(tok), u64(page)};
  const u32 box[3] = {u32(a.heads * bytes), u32(1) << a.box_log2, 1}, estr[3] = {1, 1, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Bytes of scales that can be copied at a time: 16 where a block's heads follow one another and rows are aligned.
inline int scale_unit(const Args& a, const uint8_t* base, long long page, long long tok, long long head, int bytes) {
  const int H_kv = a.cache.H_kv, last = (H_kv - 1) % a.heads + 1;
  if (H_kv == 1) head = bytes;
  const long long all = page | tok;
  if (head == bytes && aligned(base, 16) && all % 16 == 0 && a.heads * bytes % 16 == 0 && last * bytes % 16 == 0) return 16;
  return bytes == 8 && aligned(base, 8) && (all | head) % 8 == 0 ? 8 : 4;
}

// Blocks as for the wider caches: chunks of a head first (they read the same tile), then heads side by side, then runs of tokens.
template <int DQK, int DV, int NC>
bool plan4(Args& a, int nsm, int* smem) {
  using T = Tile4<DQK, DV>;
  a.chunks = (a.group + 8 * NC - 1) / (8 * NC);
  a.chunk_heads = (a.group + a.chunks - 1) / a.chunks;
  a.chunk_warps = piece(a.chunks, kWarps);
  a.heads = piece(a.cache.H_kv, kWarps / a.chunk_warps);
  a.subs = 1;
  while (a.subs * 2 * a.heads * a.chunk_warps <= kWarps) a.subs *= 2;
  a.turns = 1;
  while (a.turns * 2 * a.subs * a.heads <= kWarps) a.turns *= 2;
  a.tile_tokens = a.subs * a.turns * kKeys;
  a.tile_log2 = log2_of(a.tile_tokens);
  a.units = (a.cache.H_kv + a.heads - 1) / a.heads * ((a.chunks + a.chunk_warps - 1) / a.chunk_warps);
  const int k_pitch = a.heads * T::kRowK, v_pitch = a.heads * T::kRowV;
  a.k_log2 = share_log2(k_pitch);
  a.v_log2 = share_log2(v_pitch);
  // Keys in the order in which the rows that one phase of the reads of K takes lie in different banks: two of 64 bytes, four of 32.
  a.order = DQK >= 128 ? (a.k_log2 == 0 ? 0x73625140u : 0x76543210u) : a.k_log2 == 0 ? 0x75316420u : a.k_log2 == 1 ? 0x76325410u : 0x76543210u;
  // Boxes: as many tokens of a page as divide both the page and the tile, in whole swizzle patterns of 1 KiB.  Heads that do not
  // follow one another, rows of other widths and smaller pages come piece by piece.
  int box = a.tile_tokens;
  while (box > 1 && a.cache.page_size % box != 0) box /= 2;
  const CacheView& c = a.cache;
  a.boxes = box >= 16 && boxable(a, c.k_page, c.k_tok, c.k_head, T::kRowK, a.k_log2, box) && boxable(a, c.v_page, c.v_tok, c.v_head, T::kRowV, a.v_log2, box);
  const ScaleView& s = a.scales;
  a.k_unit = scale_unit(a, s.k, s.k_page, s.k_tok, s.k_head, T::kScaleK);
  a.v_unit = scale_unit(a, s.v, s.v_page, s.v_tok, s.v_head, T::kScaleV);
  // The scales of a box: one run of bytes where a block takes all heads, else rows of a multiple of 16 bytes.
  auto run = [&](const uint8_t* base, long long page, long long tok, long long head, int bytes) {
    return a.heads == c.H_kv && tok == a.heads * bytes && (c.H_kv == 1 || head == bytes) && aligned(base, 16) && page % 16 == 0;
  };
  a.dense = run(s.k, s.k_page, s.k_tok, s.k_head, T::kScaleK) && run(s.v, s.v_page, s.v_tok, s.v_head, T::kScaleV);
  auto spaced = [](long long page, long long tok) { return page > 0 && tok > 0 && page < (1ll << 40) && tok < (1ll << 40); };
  a.boxes = a.boxes && (a.dense || (a.k_unit == 16 && a.v_unit == 16 && spaced(s.k_page, s.k_tok) && spaced(s.v_page, s.v_tok)));
  a.box_log2 = a.boxes ? log2_of(box) : a.tile_log2;
  const int nq = a.chunks > a.chunk_warps ? a.chunk_warps * a.chunk_heads : a.heads * a.group;
  a.q_bytes = static_cast<int>(round_up(nq * DQK * 2, 16));
  const int warps = a.heads * a.chunk_warps * a.subs;
  const int stage = static_cast<int>(round_up(bytes4(a.tile_tokens, k_pitch, a.k_log2) + bytes4(a.tile_tokens, v_pitch, a.v_log2) +
                                                  a.heads * a.tile_tokens * (T::kScaleK + T::kScaleV) + a.q_bytes, 1024));
  const int meeting = a.subs > 1 ? warps * 8 * NC * (DV + 2) * 4 : 0;  // (m, l, O) of the warps that share a head's tokens
  constexpr int kStatic = 8192;  // the schedule's tables, headers and rows, with the 1 KiB that each block takes
  int blocks = NC == 1 ? 3 : 2;
  while (blocks > 1 && blocks * (2 * stage + meeting + kStatic) > kSmemPerSm) --blocks;
  a.stages = std::min(kStages, (std::min(kSmemPerSm / blocks - kStatic, kSmemPerBlock - 8192) - meeting) / stage);
  if (a.stages < 2) return false;
  const long long most = std::max(1ll, (a.max_len + a.tile_tokens - 1ll) / a.tile_tokens), at_once = std::max(1ll, static_cast<long long>(nsm) * blocks / a.units);
  const long long turns_whole = (a.B + at_once - 1) / at_once * most, turns_split = (a.B * most + at_once - 1) / at_once;
  a.whole = most <= kLongest && turns_whole - turns_split <= kSerial;
  a.groups = static_cast<int>(a.whole ? a.B : std::min({at_once, a.B * most, parts_at_most(a.B, a.H, a.cache.H_kv, a.max_len)}));
  *smem = a.stages * stage + meeting;
  return true;
}

template <int DQK, int DV, int NC>
zyfa_status_t launch4(Args& a, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  int smem;
  set_workspace(a, ws);
  if (!plan4<DQK, DV, NC>(a, nsm, &smem)) return ZYFA_ERR_UNSUPPORTED;
  Maps4 maps = {};
  const CacheView& c = a.cache;
  using T = Tile4<DQK, DV>;
  if (a.boxes && !(make_map4(&maps.k, c.k, a, c.k_page, c.k_tok, T::kRowK, a.k_log2) && make_map4(&maps.v, c.v, a, c.v_page, c.v_tok, T::kRowV, a.v_log2) &&
                   (a.dense || (make_scale_map(&maps.ks, a.scales.k, a, a.scales.k_page, a.scales.k_tok, T::kScaleK) &&
                                make_scale_map(&maps.vs, a.scales.v, a, a.scales.v_page, a.scales.v_tok, T::kScaleV))))) {
    a.boxes = 0;
    a.box_log2 = a.tile_log2;
  }
  static std::atomic<int> set[kMaxDevices];
  if (!prepare(decode4_kernel<DQK, DV, NC>, 2, dev, set)) return ZYFA_ERR_CUDA;
  if (launch_dependent(decode4_kernel<DQK, DV, NC>, dim3(static_cast<unsigned>(a.groups) * a.units), (a.heads * a.chunk_warps * a.subs + 1) * 32, smem, stream,
                       a, maps) != cudaSuccess)
    return ZYFA_ERR_CUDA;
  return a.whole ? ZYFA_OK : launch_join<DV>(a, nsm, dev, stream);
}

}  // namespace decode4
}  // namespace zyfa
