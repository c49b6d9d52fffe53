// Attention of one new token per request over a 4-bit paged cache: device code.
//
// The mathematics, the split of the work over requests, its schedule and the join are those of the e4m3 and bf16 caches
// (decode.cuh): one pass with the running maximum and sum, tiles of all requests numbered one after the other and dealt evenly, parts
// joined in order.  What differs is a tile: codes and scales come in, and are widened where they are used.
//
// * Products run with keys (or channels of V) as the rows of mma.sync.m16n8k16 and query heads as its 8 columns, in fp16: a code
//   times its scale has 6 bits and is exact there, and a bf16 query is, over a power of two near its row's largest.
// * K: ldmatrix hands a lane 4 bytes of a key, 8 neighbouring channels.  The contraction may take channels in any order, as long as the
//   queries' fragments do: each byte, converted and multiplied by its scale both channels at a time, is an operand.
// * V: the contraction runs over keys, two of which share a register, while the two codes of a byte are channels.  ldmatrix
//   transposes 16-bit elements, four channels of a key.  Two registers with the same channels of other keys exchange nibbles (4 operations
//   for 16 values), so that a byte is one channel of two keys: converted and multiplied by their scales, it is an operand.
// * Codes are numbers whatever their bits, so what lies in shared memory behind a request's end only needs scales of 0.
//
// Bound: HBM, 9/16 byte a value, and next to it the SM's issue: 16 keys of a head of 128 channels are some 318 warp instructions for 2304
// bytes, 64 of which convert, 64 multiply by scales and 16 are matrix products.  128 requests of up to 16384 tokens, 8 KV heads of 128: 134 us,
// where the bytes take 101 and the loads alone 111; 2.4 instructions a clock and SM, the ALU at half its rate, matrix instructions at a
// quarter of theirs.  More warps an SM would fill the gaps, but 96 registers a thread spill (166 us with 16 compute warps).  V's registers are
// on their way while scores become weights, which needs the queries' fragments in shared memory: 16 of 192/128 74 -> 70 us (in registers
// both spill: 142 us for the 128 requests).  Scales taken outside the matrix products, on weights and scores, cost as many instructions;
// tcgen05 would read widened operands from shared memory, which takes longer than the whole kernel.
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
  int k_each, v_each;    // boxes: rows lie in shared memory head by head, not side by side
  int ks_mode, vs_mode;  // boxes: how scales come (kRows ...)
  int k_log2, v_log2;    // tokens whose rows share 128 bytes of shared memory (log2), where a block's heads take less
  int meeting_bytes;     // of shared memory behind the stages, where warps that share a head's tokens meet; the queries' fragments follow
  int k_unit, v_unit;    // bytes of scales copied at a time: 4, 8, or 16 across heads
};

// Scales of a box as rows of [token][head] bytes by TMA, as the one run of bytes that such rows are, or as a run for each head.
enum : int { kRows, kRun, kRunEach };

struct Maps4 {
  CUtensorMap k, v, ks, vs;
};

template <int DQK, int DV>
struct Tile4 {
  static constexpr int kRowK = DQK / 2, kRowV = DV / 2, kScaleK = DQK / 16, kScaleV = DV / 16;
};

// Codes of a tile lie in shared memory box by box, a token's heads one after the other, in columns of 128 bytes [token][128] with
// the 16-byte pieces of a row exchanged by its number, as TMA's 128-byte swizzle does; rows of 32 or 64 bytes share 128 (`log2`).
//
// Heads whose rows do not follow one another (`each`) have a column of their own [token][row], with the pieces exchanged as the swizzle of
// 64 or 32 bytes does for such rows (`exchange`: 3, 1), and not at all for rows of 96 bytes.
struct Place {
  int row_bytes, log2, box_log2, exchange;
  bool each;
  uint32_t box_bytes;
  __device__ __forceinline__ uint32_t operator()(int token, int head, int byte) const {
    const int in = token & ((1 << box_log2) - 1);
    uint32_t at = (token >> box_log2) * box_bytes;
    if (each) {
      at += (head * row_bytes) << box_log2;
      if (exchange == 0) return at + in * row_bytes + byte;
    } else {
      byte += head * row_bytes;
    }
    const int row = in >> log2, inner = ((in & ((1 << log2) - 1)) << (7 - log2)) + byte;
    return at + (inner >> 7) * (128u << (box_log2 - log2)) + row * 128 + (((inner >> 4 & 7) ^ (row & exchange)) << 4) + (inner & 15);
  }
  // of a multiple of 16 tokens, from token 0
  __device__ __forceinline__ uint32_t step(int token) const {
    const int in = token & ((1 << box_log2) - 1);
    return (token >> box_log2) * box_bytes + (each && exchange == 0 ? in * row_bytes : (in >> log2) * 128);
  }
};
__host__ __device__ inline uint32_t bytes4(int tokens, int pitch, int log2) { return static_cast<uint32_t>(tokens >> log2) * 128u * ((pitch + 127) / 128); }
inline int share_log2(int pitch) { return pitch == 32 ? 2 : pitch == 64 ? 1 : 0; }

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
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t halves(float lo, float hi) { return pack2<true>(lo, hi); }

// The order of 16 keys in V's matrices and in K's.  A register of V's first matrix and the one of its second pair nibble by nibble: rows 2t of
// both, and rows 2t + 1.  Weights leave the scores' rows in pairs 2t, 2t + 1, so K's rows are these keys: those of V's two matrices in turn.
// Keys of a matrix are apart mod 8 in both, which keeps its rows in different banks.
__host__ __device__ constexpr int key_of_v(int row) { return row < 8 ? row : 8 + (row + 1) % 8; }
__host__ __device__ constexpr int key_of_k(int row) { return key_of_v((row & 1) * 8 + (row & 6) + (row >> 3)); }

// Where a lane's ldmatrix reads of a run of 32 keys go, relative to the run's first key (a multiple of 32): row (lane & 7), 8 on for the
// odd matrices, and of its 16-byte pieces one, or the next for the last two matrices.  16 keys on, the exchange of pieces is the same
// unless four tokens share a row (64 channels, one head).
template <int DQK, int DV>
struct Reader4 {
  static constexpr int kPairsK = DQK / 64, kPairsV = DV / 64;  // of 16-byte pieces, 32 channels each
  uint32_t key[DQK == 64 ? 2 : 1][kPairsK], value[DV == 64 ? 2 : 1][kPairsV];
  uint32_t k_16, v_16;               // from 16 keys to the next
  uint32_t k_scale[2];               // of rows g and g + 8 of K
  uint32_t v_scale, v_last;          // of row 2t of V's first matrix, and row 2t + 1 of its second
  uint32_t k_scales, v_scales;       // from a key's scales to the next's
  uint32_t v_zero;                   // of key `lane`

  __device__ __forceinline__ void set(const Args& a, int lane, int head, int first, const Place& kp, const Place& vp) {
    using T = Tile4<DQK, DV>;
    const int row = lane & 15, piece = (lane >> 4) * 16, k_row = first + key_of_k(row), v_row = first + key_of_v(row);
    k_16 = kp.step(16);
    v_16 = vp.step(16);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
#pragma unroll
      for (int i = 0; i < kPairsK; ++i)
        if (n == 0 || DQK == 64) key[n][i] = kp(k_row + 16 * n, head, 32 * i + piece) - n * k_16;
#pragma unroll
      for (int i = 0; i < kPairsV; ++i)
        if (n == 0 || DV == 64) value[n][i] = vp(v_row + 16 * n, head, 32 * i + piece) - n * v_16;
    }
    const bool k_each = a.boxes && a.ks_mode == kRunEach, v_each = a.boxes && a.vs_mode == kRunEach;
    k_scales = (k_each ? 1 : a.heads) * T::kScaleK;
    v_scales = (v_each ? 1 : a.heads) * T::kScaleV;
    v_zero = (first + lane) * v_scales + head * T::kScaleV * (v_each ? a.tile_tokens : 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) k_scale[j] = (first + key_of_k((lane >> 2) + 8 * j)) * k_scales + head * T::kScaleK * (k_each ? a.tile_tokens : 1);
    v_scale = v_zero + (2 * (lane & 3) - lane) * v_scales;
    v_last = v_zero + (key_of_v(2 * (lane & 3) + 9) - lane) * v_scales;
  }
  // row 2t (2t + 1) of V's first matrix (its second)
  __device__ __forceinline__ uint32_t value_scale(bool odd, bool second) const {
    return !second ? v_scale + odd * v_scales : odd ? v_last : v_scale + key_of_v(8) * v_scales;
  }
  __device__ __forceinline__ uint32_t key_at(int i, bool second) const { return DQK == 64 && second ? key[DQK == 64][i] : key[0][i]; }
  __device__ __forceinline__ uint32_t value_at(int i, bool second) const { return DV == 64 && second ? value[DV == 64][i] : value[0][i]; }
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
// the state of a compute warp: up to kHeads query heads against its tiles

// A set is 8 heads, the columns of a product; sets share the products of codes by scales.
template <int DQK, int DV, int NS>
struct Rows4 {
  using T = Tile4<DQK, DV>;
  using R = Reader4<DQK, DV>;
  static constexpr int kHeads = 8 * NS, kPiecesK = DQK / 32, kPieces = DV / 32;
  static constexpr uint32_t kQueryBytes = NS * kPiecesK * 512;  // B fragments in shared memory, a lane's of two steps of the contraction in 16 bytes
  // Runs of 16 keys whose scores are weighed together: both of a turn where registers hold them (128 requests 136 us, one by one 138; two
  // sets of 64 channels 31.1 and 33.7; two sets of 128 would spill 144 bytes a thread: 51 us instead of 45).
  static constexpr int kTogether = NS == 1 || DV == 64 ? 2 : 1;
  static constexpr float kLift = 15.0f;             // weights in fp16 up to 2^15, so that light ones keep their bits
  static constexpr float kNoKey = 3.402823466e38f;  // ref before the first key: lifts every score above its negative over the limit
  // From this magnitude of m on scores are rounded before m is subtracted.  Below, the product with `scale` and the sum with ref round as
  // one, by less than 2^-13 of a weight's exponent; from 2^24 on by whole units, which took weights out of fp16.
  static constexpr float kLoud = 1024.0f;

  uint32_t queries;
  float o[NS][kPieces][2][4], m[NS][2], l[NS][2];  // this lane's two heads of each set
  F2 ref[NS], scale[NS];
  float dv;

  __device__ __forceinline__ uint4 query(int c, int p) const { return lds16(queries + (c * kPiecesK + p) * 512); }
  static __device__ __forceinline__ uint32_t top_bits(uint32_t top, uint32_t w) { return max(top, max(w & 0x7fff0000u, (w << 16) & 0x7fff0000u)); }

  // Begins a request's part: its queries from shared memory, `count` dense bf16 rows.
  __device__ __forceinline__ void begin(uint32_t rows, int count, float scale_, float dv_, int lane) {
    const int t = lane & 3;
    __syncwarp();  // the last part's fragments have been read
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      // rows behind the last head repeat it: their columns are computed and never written
      const uint32_t row = rows + min(8 * c + (lane >> 2), count - 1) * (DQK * 2) + 16 * t;
      uint32_t top = 0;
#pragma unroll
      for (int p = 0; p < kPiecesK; ++p) {
        const uint4 w = lds16(row + 64 * p);
        top = top_bits(top_bits(top_bits(top_bits(top, w.x), w.y), w.z), w.w);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the largest magnitude to [2^14, 2^15), which an infinity or NaN stays beyond
      const int shift = min(127, 141 - static_cast<int>(top >> 23));
      const float f = __uint_as_float(static_cast<uint32_t>(127 + shift) << 23);
#pragma unroll
      for (int p = 0; p < kPiecesK; ++p) {
        const uint4 w = lds16(row + 64 * p);
        auto two = [&](uint32_t x) { return halves(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f); };
        const uint4 q = make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
        ptx::st_shared_v4(queries + (c * kPiecesK + p) * 512, q.x, q.y, q.z, q.w);
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
    __syncwarp();
  }

  // The scales of one key (of D channels) for this lane's block of each 32 channels, widened: two a register.
  template <int D>
  static __device__ __forceinline__ void scales_of(uint32_t at, bool second, uint32_t (&s)[(D / 32 + 1) / 2]) {
    if constexpr (D == 64) {
      s[0] = widen_e4m3(prmt(lds4(at), 0, second ? 0x31 : 0x20));
    } else if constexpr (D == 128) {
      const uint2 w = lds8(at);
      const uint32_t x = prmt(w.x, w.y, second ? 0x7531 : 0x6420);
      s[0] = widen_e4m3(x);
      s[1] = widen_e4m3_hi(x);
    } else {
      const uint32_t x = prmt(lds4(at), lds4(at + 4), second ? 0x7531 : 0x6420);
      s[0] = widen_e4m3(x);
      s[1] = widen_e4m3_hi(x);
      s[2] = widen_e4m3(prmt(lds4(at + 8), 0, second ? 0x31 : 0x20));
    }
  }
  // One of two fp16 numbers in both places (which a product takes as it is).
  static __device__ __forceinline__ uint32_t both(uint32_t x, int which) {
    uint32_t d;
    if (which)
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tmov.b32 %0, {hi, hi};\n\t}" : "=r"(d) : "r"(x));
    else
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tmov.b32 %0, {lo, lo};\n\t}" : "=r"(d) : "r"(x));
    return d;
  }
  static __device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%6, %7};\n\tfma.rn.f32x2 p, p, q, r;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
  }
  // The scores of 16 keys (second: of the run of 32, the second 16), over scale: rows are keys, columns heads; two chains of products.
  __device__ __forceinline__ void scores(const Run4& s, const R& at, bool second, int t, F2 (&x)[NS][2]) {
    float acc[2][NS][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < NS; ++c) acc[j][c][0] = acc[j][c][1] = acc[j][c][2] = acc[j][c][3] = 0.0f;
    const uint32_t ks = s.ks + (second ? 16 * at.k_scales : 0), k = s.k + (second ? at.k_16 : 0);
    uint32_t sa[(kPiecesK + 1) / 2], sb[(kPiecesK + 1) / 2];
    scales_of<DQK>(ks + at.k_scale[0], t >= 2, sa);
    scales_of<DQK>(ks + at.k_scale[1], t >= 2, sb);
#pragma unroll
    for (int i = 0; i < kPiecesK / 2; ++i) {
      uint32_t r[4];
      ldsm4(k + at.key_at(i, second), r);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t ka = r[2 * j], kb = r[2 * j + 1];
        const uint32_t fa = both(sa[i], j), fb = both(sb[i], j);
        const uint32_t a0 = mul_f16x2(widen_e2m1<0>(ka), fa), a1 = mul_f16x2(widen_e2m1<0>(kb), fb);
        const uint32_t a2 = mul_f16x2(widen_e2m1<1>(ka), fa), a3 = mul_f16x2(widen_e2m1<1>(kb), fb);
        const uint32_t b0 = mul_f16x2(widen_e2m1<2>(ka), fa), b1 = mul_f16x2(widen_e2m1<2>(kb), fb);
        const uint32_t b2 = mul_f16x2(widen_e2m1<3>(ka), fa), b3 = mul_f16x2(widen_e2m1<3>(kb), fb);
#pragma unroll
        for (int c = 0; c < NS; ++c) {
          const uint4 q = query(c, 2 * i + j);
          mma<kF16>(acc[0][c], a0, a1, a2, a3, q.x, q.y);
          mma<kF16>(acc[1][c], b0, b1, b2, b3, q.z, q.w);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NS; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j) x[c][j] = add2({acc[0][c][2 * j], acc[0][c][2 * j + 1]}, {acc[1][c][2 * j], acc[1][c][2 * j + 1]});
  }
  // V's matrices of 16 keys and the scales of rows 2t and 2t + 1 of both, as they lie in shared memory.
  struct Raw {
    uint32_t r[kPieces / 2][4];
    uint2 first[2], other[2];
  };
  __device__ __forceinline__ void load_values(const Run4& s, const R& at, bool second, Raw& v) const {
    const uint32_t vs = s.vs + (second ? 16 * at.v_scales : 0), v0 = s.v + (second ? at.v_16 : 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t first = vs + at.value_scale(j, false), other = vs + at.value_scale(j, true);
      v.first[j] = DV == 128 ? lds8(first) : make_uint2(lds4(first), 0);
      v.other[j] = DV == 128 ? lds8(other) : make_uint2(lds4(other), 0);
    }
#pragma unroll
    for (int p = 0; p < kPieces / 2; ++p) ldsm4t(v0 + at.value_at(p, second), v.r[p]);
  }
  // O^T += V^T P^T of 16 keys: rows are channels of V, the contraction keys.
  __device__ __forceinline__ void values(const Raw& raw, int g, const uint32_t (&pf)[NS][2]) {
    uint32_t sv[2][kPieces];  // scales of this lane's block of every 32 channels
    const uint32_t pick = g < 4 ? 0x6240u : 0x7351u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo = prmt(raw.first[j].x, raw.other[j].x, pick);
      sv[j][0] = widen_e4m3(lo);
      sv[j][1] = widen_e4m3_hi(lo);
      if constexpr (DV == 128) {
        const uint32_t hi = prmt(raw.first[j].y, raw.other[j].y, pick);
        sv[j][2] = widen_e4m3(hi);
        sv[j][3] = widen_e4m3_hi(hi);
      }
    }
#pragma unroll
    for (int p = 0; p < kPieces; p += 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // two keys a byte: even channels, and odd ones
        const uint32_t v = raw.r[p / 2][2 * i], w = raw.r[p / 2][2 * i + 1];
        const uint32_t even = (v & 0x0f0f0f0fu) | (w << 4 & 0xf0f0f0f0u), odd = (v >> 4 & 0x0f0f0f0fu) | (w & 0xf0f0f0f0u);
        const uint32_t s0 = sv[0][p + i], s1 = sv[1][p + i];
        const uint32_t f[2][4] = {{mul_f16x2(widen_e2m1<0>(even), s0), mul_f16x2(widen_e2m1<0>(odd), s0), mul_f16x2(widen_e2m1<1>(even), s0),
                                   mul_f16x2(widen_e2m1<1>(odd), s0)},
                                  {mul_f16x2(widen_e2m1<2>(even), s1), mul_f16x2(widen_e2m1<2>(odd), s1), mul_f16x2(widen_e2m1<3>(even), s1),
                                   mul_f16x2(widen_e2m1<3>(odd), s1)}};
#pragma unroll
        for (int c = 0; c < NS; ++c) {
          mma<kF16>(o[c][p + i][0], f[0][0], f[0][1], f[1][0], f[1][1], pf[c][0], pf[c][1]);
          mma<kF16>(o[c][p + i][1], f[0][2], f[0][3], f[1][2], f[1][3], pf[c][0], pf[c][1]);
        }
      }
    }
  }

  // One run of 32 keys.  FULL: all count; else mask: those that do, at least one.
  template <bool FULL>
  __device__ __forceinline__ void tile(const Run4& s, const R& at, uint32_t mask, int lane) {
    if constexpr (kTogether == 2) {
      weigh<FULL>(s, at, 0, mask, lane);
    } else {
#pragma unroll 1
      for (int i = 0; i < 2; ++i) weigh<FULL>(s, at, i, mask >> (16 * i), lane);
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void weigh(const Run4& s, const R& at, int from, uint32_t mask, int lane) {
    constexpr int H = kTogether;
    const int g = lane >> 2, t = lane & 3;
    F2 x[H][NS][2];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      scores(s, at, from + h, t, x[h]);
      if (!FULL)
#pragma unroll
        for (int c = 0; c < NS; ++c)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            x[h][c][j] = mul2(x[h][c][j], scale[c]);
            if (!((mask >> (16 * h + key_of_k(j * 8 + g))) & 1)) x[h][c][j] = {-INFINITY, -INFINITY};
          }
    }
    Raw raw;  // on its way while scores become weights
    load_values(s, at, from, raw);
    uint32_t pf[H][NS][2];
#pragma unroll
    for (int c = 0; c < NS; ++c) {
      // log2 of the weights: scores in units of log2 over the reference m, which moves only when a key exceeds it: log2 of a weight is then
      // above the lift.  A loud m leaves ref at kNoKey, so that every run comes by here.
      F2 y[H][2];
      float over;
      auto log2_weights = [&]() {
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            y[h][j] = FULL ? fma2(scale[c], x[h][c][j], ref[c]) : add2(x[h][c][j], ref[c]);
            const float top = fmaxf(y[h][j].x, y[h][j].y);
            over = h + j ? fmaxf(over, top) : top;
          }
      };
      log2_weights();
      if (__any_sync(0xffffffffu, over > kLift)) {
        // (rounded by itself; products, since a descale below 0 turns the order of sums around)
        auto score = [&](int h, int j, int e) {
          const float s = e ? x[h][c][j].y : x[h][c][j].x;
          return FULL ? __fmul_rn(e ? scale[c].y : scale[c].x, s) : s;
        };
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = m[c][e];
#pragma unroll
          for (int h = 0; h < H; ++h) top = fmaxf(top, fmaxf(score(h, 0, e), score(h, 1, e)));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float f = top == -INFINITY ? 1.0f : exp2_approx(m[c][e] - top);
          m[c][e] = top;
          (e ? ref[c].y : ref[c].x) = fabsf(top) < kLoud ? kLift - top : kNoKey;
          l[c][e] *= f;
#pragma unroll
          for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              o[c][i][j][e] *= f;
              o[c][i][j][e + 2] *= f;
            }
        }
        log2_weights();
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (fabsf(m[c][e]) >= kLoud && m[c][e] != -INFINITY)
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int j = 0; j < 2; ++j) (e ? y[h][j].y : y[h][j].x) = (score(h, j, e) - m[c][e]) + kLift;  // the greatest one's is the lift
      }
      // Weights, transposed into the B operand (keys are now the contraction).  They round to the 11 bits of fp16, by an eighth
      // of what out rounds by at most, beside a V that fp16 holds exactly; two terms would double the products.  Their sum takes them unrounded.
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const F2 w = {exp2_approx(y[h][j].x), exp2_approx(y[h][j].y)};
          const F2 sum = add2({l[c][0], l[c][1]}, w);
          l[c][0] = sum.x;
          l[c][1] = sum.y;
          pf[h][c][j] = transpose8x8(halves(w.x, w.y));
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const Raw now = raw;
      if (h + 1 < H) load_values(s, at, from + h + 1, raw);
      values(now, g, pf[h]);
    }
  }

  // Ends a request's part: writes its rows (`count` query heads from `first`), or (m, l, O) to part `slot` of the workspace.
  __device__ __forceinline__ void finish(const DecodeArgs& a, int b, int first, int count, bool direct, long long slot, int lane) {
    const int g = lane >> 2;
#pragma unroll
    for (int c = 0; c < NS; ++c)
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
  // all_ml, all_o: [subs][kHeads] and [subs][kHeads][DV], `stride` warps from one sub's to the next; meet() is false if it gave up.
  template <typename F>
  __device__ __forceinline__ bool finish_shared(const DecodeArgs& a, int b, int first, int count, bool direct, long long slot, int lane, int sub,
                                                int subs, int stride, float2* all_ml, float* all_o, F meet) {
    const int g = lane >> 2;
    float2* my_ml = all_ml + sub * stride * kHeads;
    float* my_o = all_o + sub * stride * kHeads * DV;
#pragma unroll
    for (int c = 0; c < NS; ++c)
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
// what both kernels share: a block's part of the work, its memory, its compute warps

template <int NS>
constexpr int kBlocks = NS == 1 ? 3 : 2;  // an SM

template <int DQK, int DV>
struct Block4 {
  using T = Tile4<DQK, DV>;
  const Args& a;
  const int lane, warp;
  // a stage: K, V, scales of K, scales of V, queries
  uint32_t k_bytes, ks_at, vs_at, q_at, stage_bytes, tiles, full, empty;
  Place k_place, v_place;
  unsigned g;                        // this block's group ...
  int head0, chunk0, chunk_units;    // ... KV heads from head0, chunks of query heads from chunk0
  int b, left;                       // and run: first request, numbers (0: none), and the first tile of it
  unsigned tile0;

  __device__ __forceinline__ Block4(const Args& a_, uint8_t* smem, uint64_t* full_, uint64_t* empty_) : a(a_), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {
    const int TT = a.tile_tokens, k_pitch = a.heads * T::kRowK, v_pitch = a.heads * T::kRowV;
    k_bytes = bytes4(TT, k_pitch, a.k_log2);  // (no less than rows head by head take)
    ks_at = k_bytes + bytes4(TT, v_pitch, a.v_log2);
    vs_at = ks_at + a.heads * TT * T::kScaleK;
    q_at = vs_at + a.heads * TT * T::kScaleV;
    stage_bytes = (q_at + a.q_bytes + 1023) & ~1023u;
    auto place = [&](int row, int pitch, int log2, bool each) {
      if (!each) return Place{row, log2, a.box_log2, 7, false, bytes4(1 << a.box_log2, pitch, log2)};
      return Place{row, row == 64 ? 1 : row == 32 ? 2 : 0, a.box_log2, row == 64 ? 3 : row == 32 ? 1 : 0, true, static_cast<uint32_t>(pitch) << a.box_log2};
    };
    k_place = place(T::kRowK, k_pitch, a.k_log2, a.boxes && a.k_each);
    v_place = place(T::kRowV, v_pitch, a.v_log2, a.boxes && a.v_each);
    tiles = smem_addr(smem);
    full = smem_addr(full_);
    empty = smem_addr(empty_);
    g = blockIdx.x / a.units;
    const int unit = blockIdx.x % a.units;
    chunk_units = (a.chunks + a.chunk_warps - 1) / a.chunk_warps;
    head0 = unit / chunk_units * a.heads;
    chunk0 = unit % chunk_units * a.chunk_warps;
  }
  __device__ __forceinline__ void init_barriers(uint64_t* meet, int full_count, int warps) const {
    for (int i = 0; i < a.stages; ++i) {
      ptx::mbar_init(full + 8 * i, full_count);
      ptx::mbar_init(empty + 8 * i, warps);
    }
    for (int i = 0; i < a.heads * a.chunk_warps; ++i) ptx::mbar_init(smem_addr(meet + i), a.subs);
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  __device__ __forceinline__ void find(unsigned* prefix, unsigned* sums) {
    if (a.whole) {
      b = static_cast<int>(g);
      tile0 = 0;
      left = static_cast<int>(Schedule::tiles(a, b));
    } else {
      Schedule plan;
      plan.find(a, prefix, sums, true, g, &b, &tile0, &left);
    }
  }
  __device__ __forceinline__ void write_empty(int q0, int nq) const {
    const long long row = static_cast<long long>(b) * a.H + q0;
    for (int i = lane; i < nq * DV / 2; i += 32) reinterpret_cast<__nv_bfloat162*>(a.out + row * DV)[i] = __floats2bfloat162_rn(0.0f, 0.0f);
    if (a.lse)
      for (int i = lane; i < nq; i += 32) a.lse[row + i] = -INFINITY;
  }
  __device__ __forceinline__ int heads() const { return min(a.heads, a.cache.H_kv - head0); }
  // The scales of the scores and of V of a request that begins with a tile.
  __device__ __forceinline__ void descales(int request, float2* to) const {
    if (lane < heads()) {
      const int i = a.desc_per_head ? request * a.desc_request + head0 + lane : 0;
      to[lane] = {a.scale_log2 * (a.k_desc ? a.k_desc[i] : 1.0f), a.v_desc ? a.v_desc[i] : 1.0f};
    }
  }
  // One lane: what the compute warps need to know of a tile, and its queries; `bytes` of other copies count on the barrier.
  __device__ __forceinline__ void publish(Header* header, const Cursor& c, int st, int valid, bool whole, uint32_t bytes) const {
    const uint32_t bar = full + 8 * st;
    *header = {c.b, c.flags(a.tile_tokens) | (whole ? 0 : kPartial), valid, 0};
    if (c.first) {
      // the block's query rows: whole heads, or (more chunks than warps) part of one head's
      const int first_q = head0 * a.group + chunk0 * a.chunk_heads;
      const uint32_t rows = chunk_units > 1 ? min(a.chunk_warps * a.chunk_heads, a.group - chunk0 * a.chunk_heads) : heads() * a.group;
      bulk_load(tiles + st * stage_bytes + q_at, a.q + c.b * a.q_batch + static_cast<long long>(first_q) * (DQK * 2), rows * (DQK * 2), bar);
      bytes += rows * (DQK * 2);
    }
    ptx::mbar_arrive_expect_tx(bar, bytes);
  }
};

// mbar_wait_bounded whose usual case, a phase that has ended, is a few instructions.
__device__ __forceinline__ bool wait4(uint32_t bar, uint32_t parity, long long clocks) {
  return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)) || mbar_wait_bounded(bar, parity, clocks);
}

// A compute warp's way through the block's tiles.
// ZERO: the scales of V that belong to no key are to be cleared.
template <typename Rows, int DQK, int DV, bool ZERO>
__device__ __forceinline__ void compute4(const Block4<DQK, DV>& k, uint8_t* smem, const Header* headers, const float2 (*scales)[kWarps], const unsigned (*masks)[kWarps],
                                         uint64_t* meets, int warps) {
  using T = Tile4<DQK, DV>;
  const Args& a = k.a;
  const int lane = k.lane, warp = k.warp, S = a.stages;
  // a run of keys, a KV head, a chunk of its query heads
  const int head = warp % a.heads, chunk = k.chunk0 + warp / a.heads % a.chunk_warps, sub = warp / (a.heads * a.chunk_warps);
  const int hk = k.head0 + head, q0 = hk * a.group + chunk * a.chunk_heads, nq = min(a.chunk_heads, a.group - chunk * a.chunk_heads);
  const bool idle = hk >= a.cache.H_kv || nq <= 0;  // the last block of a group may have heads or chunks too many
  if (k.left == 0) {
    if (a.whole && sub == 0 && !idle) k.write_empty(q0, nq);  // a request without tokens
    return;
  }
  Reader4<DQK, DV> reader;
  const int run_keys = a.turns * kKeys;
  reader.set(a, lane, head, sub * run_keys, k.k_place, k.v_place);
  const uint32_t my_query = k.q_at + (head * a.group + (chunk - k.chunk0) * a.chunk_heads) * (DQK * 2);
  // where warps that share a head's tokens meet
  const int peers = a.heads * a.chunk_warps, peer = warp % peers;
  uint8_t* meeting = smem + S * k.stage_bytes;
  float2* all_ml = reinterpret_cast<float2*>(meeting) + peer * Rows::kHeads;
  float* all_o = reinterpret_cast<float*>(meeting + warps * Rows::kHeads * 8) + peer * Rows::kHeads * DV;
  const uint32_t meet_s = smem_addr(meets + peer);
  uint32_t meet_parity = 0;
  // Copies still in flight write to this block's shared memory: waits for them, again for a bounded time.
  auto give_up = [&](int st, uint32_t par) {
    for (int j = 1; j < S; ++j) {
      if (++st == S) {
        st = 0;
        par ^= 1;
      }
      mbar_wait_bounded(k.full + 8 * st, par, a.wait_clocks);
    }
    if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
  };
  Rows rows;
  rows.queries = smem_addr(meeting) + a.meeting_bytes + warp * Rows::kQueryBytes + lane * 16;
  auto run_at = [&](uint32_t base, int turn) {
    Run4 s = {base, base + k.k_bytes, base + k.ks_at, base + k.vs_at};
    if (turn) {
      s.k += k.k_place.step(turn * kKeys);
      s.v += k.v_place.step(turn * kKeys);
      s.ks += turn * kKeys * reader.k_scales;
      s.vs += turn * kKeys * reader.v_scales;
    }
    return s;
  };
  int stage = 0;
  uint32_t parity = 0, base = k.tiles;
  while (true) {
    if (!wait4(k.full + 8 * stage, parity, a.wait_clocks)) {
      give_up(stage, parity);
      return;
    }
    const int flags = headers[stage].flags;
    if (flags == 0 && !idle) {  // amid a request
      for (int turn = 0; turn < a.turns; ++turn) rows.template tile<true>(run_at(base, turn), reader, 0xffffffffu, lane);
    } else if (!idle) {
      if (flags & kFirst) rows.begin(base + my_query, nq, scales[stage][head].x, scales[stage][head].y, lane);
      for (int turn = 0; turn < a.turns; ++turn) {
        const uint32_t mask = flags & kPartial ? masks[stage][sub * a.turns + turn] : 0xffffffffu;
        if (mask == 0) continue;
        const Run4 s = run_at(base, turn);
        if (ZERO && mask != 0xffffffffu) {
          // whatever the scales of keys that do not count hold is no number to multiply by 0
          const uint32_t mine = s.vs + reader.v_zero;
          if (!((mask >> lane) & 1))
#pragma unroll
            for (int i = 0; i < T::kScaleV; i += 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(mine + i), "r"(0) : "memory");
          ptx::fence_proxy_async_smem();  // before a later TMA load into this stage
          __syncwarp();
        }
        rows.template tile<false>(s, reader, mask, lane);
      }
      if (flags & kLast) {
        const bool direct = flags & kDirect;
        const int b = headers[stage].b;
        const long long slot = static_cast<long long>(k.g) * 2 + (flags & kSlot1 ? 1 : 0);
        if (a.subs == 1) {
          rows.finish(a, b, q0, nq, direct, slot, lane);
        } else {
          const bool met = rows.finish_shared(a, b, q0, nq, direct, slot, lane, sub, a.subs, peers, all_ml, all_o, [&]() {
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
    if (flags & kEnd) return;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(k.empty + 8 * stage);
    base += k.stage_bytes;
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
      base = k.tiles;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// tiles by TMA, box by box; a warp of its own issues the copies

template <int DQK, int DV, int NS>
__global__ void __launch_bounds__((kWarps + 1) * 32, kBlocks<NS>) boxes4_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps4 maps) {
  using T = Tile4<DQK, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ unsigned s_prefix[(kWarps + 1) * 32], s_sums[kWarps + 1];
  __shared__ __align__(16) Header s_header[kStages];
  __shared__ float2 s_scale[kStages][kWarps];  // of the scores, and of V
  __shared__ unsigned s_mask[kStages][kWarps]; // a tile's keys that count, 32 a word
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_meet[kWarps];
  const int warps = (blockDim.x >> 5) - 1;  // compute warps; the next one loads
  Block4<DQK, DV> k(a, smem, s_full, s_empty);
  const int lane = k.lane;
  if (threadIdx.x == 0) k.init_barriers(s_meet, 1, warps);
  if (threadIdx.x == 32) {
    ptx::tma_prefetch_desc(&maps.k);
    ptx::tma_prefetch_desc(&maps.v);
    if (a.ks_mode == kRows) ptx::tma_prefetch_desc(&maps.ks);
    if (a.vs_mode == kRows) ptx::tma_prefetch_desc(&maps.vs);
  }
  __syncthreads();
  wait_for_predecessor();
  if (!a.whole) let_successor_start();  // to the join
  k.find(s_prefix, s_sums);
  if (k.warp < warps) {
    compute4<Rows4<DQK, DV, NS>, DQK, DV, true>(k, smem, s_header, s_scale, s_mask, s_meet, warps);
    return;
  }
  if (a.stalled || k.left == 0) return;
  Cursor c;
  c.start(a, k.b, k.tile0, k.left);
  const int TT = a.tile_tokens, boxes = TT >> a.box_log2;
  const uint32_t ks_bytes = a.heads * T::kScaleK << a.box_log2, vs_bytes = a.heads * T::kScaleV << a.box_log2;
  const uint32_t all_boxes = 0xffffffffu >> (32 - boxes);
  // where a block's heads begin in the maps, and the tokens that share a row there
  const int k_column = a.k_each ? k.head0 : a.k_log2 ? 0 : k.head0 * T::kRowK / 128, v_column = a.v_each ? k.head0 : a.v_log2 ? 0 : k.head0 * T::kRowV / 128;
  const int k_share = a.k_each ? 0 : a.k_log2, v_share = a.v_each ? 0 : a.v_log2, heads = k.heads();
  // (runs for each head: those that there are)
  const uint32_t expected = k.k_place.box_bytes + k.v_place.box_bytes + (a.ks_mode == kRunEach ? heads * T::kScaleK << a.box_log2 : ks_bytes) +
                            (a.vs_mode == kRunEach ? heads * T::kScaleV << a.box_log2 : vs_bytes);
  // The scales of box n, from page pg and place off on.
  auto load_scales = [&](int mode, const CUtensorMap* map, const uint8_t* from, long long page, long long tok, long long head, int each, uint32_t to, int n, int pg,
                         int off, uint32_t bar) {
    const uint32_t all = a.heads * each << a.box_log2, one = each << a.box_log2;
    if (mode == kRows) {
      tma_load_3d(to + n * all, map, bar, k.head0 * each, off, pg);
    } else if (mode == kRun) {
      bulk_load(to + n * all, from + pg * page + off * tok, all, bar);
    } else {
      for (int h = 0; h < heads; ++h) bulk_load(to + h * TT * each + n * one, from + pg * page + off * tok + (k.head0 + h) * head, one, bar);
    }
  };
  // The pages of 32 boxes of the request at a time, a lane each (a tile's boxes are among one such 32), and the next 32 or the first of the
  // next request.
  auto pages_of = [&](int request, int len, int box0) {
    const int t = (box0 + lane) << a.box_log2;
    if (t >= len) return -1;
    int p, off;
    page_of(a, t, &p, &off);
    return a.table[request * a.table_stride + p];
  };
  int pages = pages_of(c.b, c.len, c.t >> a.box_log2 & ~31), next_b = 0, next_len = 0, next_pages = -1;
  auto look_ahead = [&](bool new_request) {
    if (new_request) {
      next_len = 0;
      if (((c.len - c.t + TT - 1) >> a.tile_log2) + static_cast<int>(kGap) < c.left)  // the run goes on behind this request
        for (next_b = c.b + 1; next_b < a.B && next_len == 0; ++next_b) next_len = length_of(a, next_b);
      --next_b;
    }
    const int box0 = (c.t >> a.box_log2 & ~31) + 32;
    next_pages = box0 << a.box_log2 < c.len ? pages_of(c.b, c.len, box0) : next_len > 0 ? pages_of(next_b, next_len, 0) : -1;
  };
  bool bad = false, begun = false;
  int stage = 0;
  uint32_t parity = 1, base = k.tiles;  // a new barrier counts as one whose phase before its first has ended
  while (true) {
    if (!wait4(k.empty + 8 * stage, parity, a.wait_clocks)) {
      if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
      break;
    }
    const uint32_t bar = k.full + 8 * stage;
    const int valid = min(TT, c.len - c.t), row = lane << a.box_log2;
    const int pg = __shfl_sync(0xffffffffu, pages, (c.t >> a.box_log2 & 31) + lane);  // of this lane's box of the tile
    const bool inside = lane < boxes && row < valid, ok = inside && pg >= 0 && pg < a.cache.num_pages;
    bad |= inside && !ok;
    const unsigned there = __ballot_sync(0xffffffffu, ok);
    if (ok) {  // (the barrier's phase cannot end before the arrival below)
      int p, off;
      page_of(a, c.t + row, &p, &off);
      tma_load_5d(base + lane * k.k_place.box_bytes, &maps.k, bar, 0, off >> k_share, k_column, 0, pg);
      tma_load_5d(base + k.k_bytes + lane * k.v_place.box_bytes, &maps.v, bar, 0, off >> v_share, v_column, 0, pg);
      load_scales(a.ks_mode, &maps.ks, a.scales.k, a.scales.k_page, a.scales.k_tok, a.scales.k_head, T::kScaleK, base + k.ks_at, lane, pg, off, bar);
      load_scales(a.vs_mode, &maps.vs, a.scales.v, a.scales.v_page, a.scales.v_tok, a.scales.v_head, T::kScaleV, base + k.vs_at, lane, pg, off, bar);
    }
    const bool whole = valid == TT && there == all_boxes;
    if (!whole)
      for (int i = 0; i < TT / 32; ++i) {
        const int r = 32 * i + lane;
        const unsigned mask = __ballot_sync(0xffffffffu, r < valid && (there >> (r >> a.box_log2) & 1));
        if (lane == 0) s_mask[stage][i] = mask;
      }
    if (c.first) k.descales(c.b, s_scale[stage]);
    __syncwarp();
    if (lane == 0) k.publish(&s_header[stage], c, stage, valid, whole, __popc(there) * expected);
    if (!begun) look_ahead(true);
    begun = true;
    const bool ended = c.ends(TT);
    c.left = c.left_after(TT);
    if (c.left <= 0) break;
    c.first = false;
    c.t += TT;
    if (ended) {
      c.b = next_b;
      c.len = next_len;
      c.t = 0;
      c.first = c.from_start = true;
    }
    if (ended || (c.t >> a.box_log2 & 31) == 0) {
      pages = next_pages;
      look_ahead(ended);
    }
    base += k.stage_bytes;
    if (++stage == a.stages) {
      stage = 0;
      parity ^= 1;
      base = k.tiles;
    }
  }
  if (bad) atomicOr(a.status, kStatusBadPageBit);
}

// ------------------------------------------------------------------------------------------------
// tiles by cp.async, piece by piece: any page size, any stride; a warp of its own loads them

template <int DQK, int DV, int NS>
__global__ void __launch_bounds__((kWarps + 1) * 32, kBlocks<NS>) pieces4_kernel(const __grid_constant__ Args a) {
  using T = Tile4<DQK, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ unsigned s_prefix[(kWarps + 1) * 32], s_sums[kWarps + 1];
  __shared__ __align__(16) Header s_header[kStages];
  __shared__ float2 s_scale[kStages][kWarps];  // of the scores, and of V
  __shared__ long long s_row[4][kMaxTokens];   // where a tile's tokens lie in the scales of K and V, and in K and V; below 0: nowhere
  __shared__ unsigned s_mask[kStages][kWarps]; // a tile's keys that count, 32 a word
  __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_meet[kWarps];
  const int warps = (blockDim.x >> 5) - 1;  // compute warps; the next one loads
  Block4<DQK, DV> b4(a, smem, s_full, s_empty);
  const int lane = b4.lane, S = a.stages, TT = a.tile_tokens;
  if (threadIdx.x == 0) b4.init_barriers(s_meet, 33, warps);  // each lane's copies, and the header
  __syncthreads();
  wait_for_predecessor();
  if (!a.whole) let_successor_start();  // to the join
  b4.find(s_prefix, s_sums);
  if (b4.warp < warps) {
    compute4<Rows4<DQK, DV, NS>, DQK, DV, false>(b4, smem, s_header, s_scale, s_mask, s_meet, warps);
    return;
  }
  if (a.stalled || b4.left == 0) return;
  const int heads = b4.heads(), head0 = b4.head0;
  Cursor c;
  c.start(a, b4.b, b4.tile0, b4.left);
  const uint8_t *k = a.cache.k + head0 * a.cache.k_head, *v = a.cache.v + head0 * a.cache.v_head;
  const uint8_t *ks = a.scales.k + head0 * a.scales.k_head, *vs = a.scales.v + head0 * a.scales.v_head;
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
  bool bad = false;
  int stage = 0;
  uint32_t parity = 1;  // a new barrier counts as one whose phase before its first has ended
  while (true) {
    if (!mbar_wait_bounded(b4.empty + 8 * stage, parity, a.wait_clocks)) {
      if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
      break;
    }
    const uint32_t base = b4.tiles + stage * b4.stage_bytes;
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
      s_row[0][32 * i + lane] = ok ? page * a.scales.k_page + at * a.scales.k_tok : -1;
      s_row[1][32 * i + lane] = ok ? page * a.scales.v_page + at * a.scales.v_tok : -1;
      s_row[2][32 * i + lane] = ok ? page * a.cache.k_page + at * a.cache.k_tok : -1;
      s_row[3][32 * i + lane] = ok ? page * a.cache.v_page + at * a.cache.v_tok : -1;
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
        if (row >= 0) copy16(to + place(r, p / kPieces, p % kPieces * 16), from + row + p / kPieces * head_stride + p % kPieces * 16, 16);
        r += step;
        p += rest;
        if (p >= all) {
          p -= all;
          ++r;
        }
      }
    };
    codes(std::integral_constant<int, T::kRowK / 16>(), s_row[2], k, a.cache.k_head, base, b4.k_place);
    codes(std::integral_constant<int, T::kRowV / 16>(), s_row[3], v, a.cache.v_head, base + b4.k_bytes, b4.v_place);
    // scales [token][head]: zeros where there is no token
    k_scales.copy(s_row[0], TT, base + b4.ks_at);
    v_scales.copy(s_row[1], TT, base + b4.vs_at);
    if (c.first) b4.descales(c.b, s_scale[stage]);
    arrive_after_copies(b4.full + 8 * stage);
    __syncwarp();
    if (lane == 0) b4.publish(&s_header[stage], c, stage, valid, whole, 0);
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
}

// ------------------------------------------------------------------------------------------------
// host side

inline bool spaced(long long stride) { return stride > 0 && stride < (1ll << 40); }

// A cache's codes (strides in bytes) as boxes of `box` tokens of a block's heads: 0 not at all, 1 rows side by side, 2 head by head.
inline int box_mode(const Args& a, long long page, long long tok, long long head, int row, int log2, int box) {
  const int H_kv = a.cache.H_kv, pitch = a.heads * row;
  if (box < 8 || !spaced(page) || !spaced(tok) || (H_kv > 1 && !spaced(head))) return 0;
  if (H_kv == 1 || head == row) {
    if (log2 > 0 && a.heads == H_kv && tok == pitch && box * pitch % 1024 == 0) return 1;  // tokens one after the other
    if (log2 == 0 && pitch % 128 == 0 && H_kv * row % 128 == 0) return 1;
  }
  return 2;
}

// The map of such boxes: [page][128-byte column][token][128], or of rows of 128 bytes that several tokens share, or [page][head][token][row].
inline bool make_map4(CUtensorMap* m, const uint8_t* base, const Args& a, long long page, long long tok, long long head, int row, int log2, bool each) {
  using u64 = cuuint64_t;
  using u32 = cuuint32_t;
  const CacheView& c = a.cache;
  if (c.H_kv == 1) head = row;
  const u32 tokens = u32(1) << a.box_log2, estr[5] = {1, 1, 1, 1, 1};
  if (each) {
    const u64 dims[5] = {u64(row), u64(c.page_size), u64(c.H_kv), 1, u64(c.num_pages)}, strides[4] = {u64(tok), u64(head), u64(tok), u64(page)};
    const u32 box[5] = {u32(row), tokens, u32(a.heads), 1, 1};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<uint8_t*>(base), dims, strides, box, estr,
                             row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : row == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  const u64 dims[5] = {128, u64(c.page_size >> log2), u64(log2 ? 1 : c.H_kv * row / 128), 1, u64(c.num_pages)};
  const u64 strides[4] = {u64(log2 ? 128 : tok), 128, u64(log2 ? 128 : tok), u64(page)};
  const u32 box[5] = {128, tokens >> log2, u32(log2 ? 1 : a.heads * row / 128), 1, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<uint8_t*>(base), dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
}

// How a box's scales come, or -1: copies of 16 bytes that a block's heads do not fill go piece by piece (dense caches [page][token][head] of 5
// KV heads: 64 requests of 500 to 8000 tokens of 128 channels 127 us, of 6 heads by boxes 41).
inline int scale_mode(const Args& a, const uint8_t* base, long long page, long long tok, long long head, int bytes) {
  const int H_kv = a.cache.H_kv, last = (H_kv - 1) % a.heads + 1;
  if (!aligned(base, 16) || page % 16 != 0 || page < 0 || tok <= 0) return -1;
  const bool follow = H_kv == 1 || head == bytes;
  if (follow && a.heads == H_kv && tok == a.heads * bytes) return kRun;
  if (follow && spaced(page) && spaced(tok) && tok % 16 == 0 && a.heads * bytes % 16 == 0 && last * bytes % 16 == 0) return kRows;
  return tok == bytes && head % 16 == 0 ? kRunEach : -1;
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
template <int DQK, int DV, int NS>
bool plan4(Args& a, int nsm, int* smem) {
  using T = Tile4<DQK, DV>;
  using Rows = Rows4<DQK, DV, NS>;
  if (a.cache.num_pages == 1) a.cache.k_page = a.cache.v_page = a.scales.k_page = a.scales.v_page = 16;  // never taken; what maps can have
  a.chunks = (a.group + Rows::kHeads - 1) / Rows::kHeads;
  a.chunk_heads = (a.group + a.chunks - 1) / a.chunks;
  a.chunk_warps = piece(a.chunks, kWarps);
  a.heads = piece(a.cache.H_kv, kWarps / a.chunk_warps);
  if (a.heads == 3 && a.cache.H_kv % 2 == 0) a.heads = 2;  // rows of two heads fill whole columns, and two runs of tokens the warps
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
  // Boxes: as many tokens of a page as divide both the page and the tile, 8 at least, in whole swizzle patterns.  Smaller pages and odd
  // strides come piece by piece.
  int box = a.tile_tokens;
  while (box > 1 && a.cache.page_size % box != 0) box /= 2;
  const CacheView& c = a.cache;
  const int k_mode = box_mode(a, c.k_page, c.k_tok, c.k_head, T::kRowK, a.k_log2, box), v_mode = box_mode(a, c.v_page, c.v_tok, c.v_head, T::kRowV, a.v_log2, box);
  a.k_each = k_mode == 2;
  a.v_each = v_mode == 2;
  const ScaleView& s = a.scales;
  a.k_unit = scale_unit(a, s.k, s.k_page, s.k_tok, s.k_head, T::kScaleK);
  a.v_unit = scale_unit(a, s.v, s.v_page, s.v_tok, s.v_head, T::kScaleV);
  a.ks_mode = scale_mode(a, s.k, s.k_page, s.k_tok, s.k_head, T::kScaleK);
  a.vs_mode = scale_mode(a, s.v, s.v_page, s.v_tok, s.v_head, T::kScaleV);
  a.boxes = k_mode && v_mode && a.ks_mode >= 0 && a.vs_mode >= 0;
  a.box_log2 = a.boxes ? log2_of(box) : a.tile_log2;
  const int nq = a.chunks > a.chunk_warps ? a.chunk_warps * a.chunk_heads : a.heads * a.group;
  a.q_bytes = static_cast<int>(round_up(nq * DQK * 2, 16));
  const int warps = a.heads * a.chunk_warps * a.subs;
  const int stage = static_cast<int>(round_up(bytes4(a.tile_tokens, k_pitch, a.k_log2) + bytes4(a.tile_tokens, v_pitch, a.v_log2) +
                                                  a.heads * a.tile_tokens * (T::kScaleK + T::kScaleV) + a.q_bytes, 1024));
  a.meeting_bytes = a.subs > 1 ? warps * Rows::kHeads * (DV + 2) * 4 : 0;  // (m, l, O)
  const int more = a.meeting_bytes + warps * static_cast<int>(Rows::kQueryBytes);
  const int kStatic = a.boxes ? 2560 : 8192;  // the schedule's tables, headers and rows, with the 1 KiB that each block takes
  int blocks = kBlocks<NS>;
  while (blocks > 1 && blocks * (2 * stage + more + kStatic) > kSmemPerSm) --blocks;
  a.stages = std::min(kStages, (std::min(kSmemPerSm / blocks - kStatic, kSmemPerBlock - 8192) - more) / stage);
  if (a.stages < 2) return false;
  const long long most = std::max(1ll, (a.max_len + a.tile_tokens - 1ll) / a.tile_tokens), at_once = std::max(1ll, static_cast<long long>(nsm) * blocks / a.units);
  const long long turns_whole = (a.B + at_once - 1) / at_once * most, turns_split = (a.B * most + at_once - 1) / at_once;
  // The wider caches' rule, whose both sides for this kernel are (2 heads of 64, 256 tokens each, in a graph): 4 requests 8.4 us whole and 8.5
  // split, 16 8.4 and 8.4, 64 8.5 and 9.3, 256 9.7 and 13.4.  One alone takes 8.4 and 7.3, but called from a host that launches twice 8.4
  // and 8.7.
  a.whole = most <= kLongest && turns_whole - turns_split <= kSerial;
  a.groups = static_cast<int>(a.whole ? a.B : std::min({at_once, a.B * most, parts_at_most(a.B, a.H, a.cache.H_kv, a.max_len)}));
  *smem = a.stages * stage + more;
  return true;
}

template <int DQK, int DV, int NS>
zyfa_status_t launch4_as(Args& a, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  int smem;
  set_workspace(a, ws);
  if (!plan4<DQK, DV, NS>(a, nsm, &smem)) return ZYFA_ERR_UNSUPPORTED;
  Maps4 maps = {};
  const CacheView& c = a.cache;
  using T = Tile4<DQK, DV>;
  const ScaleView& v = a.scales;
  if (a.boxes && !(make_map4(&maps.k, c.k, a, c.k_page, c.k_tok, c.k_head, T::kRowK, a.k_log2, a.k_each) &&
                   make_map4(&maps.v, c.v, a, c.v_page, c.v_tok, c.v_head, T::kRowV, a.v_log2, a.v_each) &&
                   (a.ks_mode != kRows || make_scale_map(&maps.ks, v.k, a, v.k_page, v.k_tok, T::kScaleK)) &&
                   (a.vs_mode != kRows || make_scale_map(&maps.vs, v.v, a, v.v_page, v.v_tok, T::kScaleV)))) {
    a.boxes = 0;
    a.box_log2 = a.tile_log2;
  }
  static std::atomic<int> set[2][kMaxDevices];
  const dim3 grid(static_cast<unsigned>(a.groups) * a.units);
  const unsigned threads = a.heads * a.chunk_warps * a.subs * 32;
  cudaError_t e;
  if (a.boxes) {
    if (!prepare(boxes4_kernel<DQK, DV, NS>, 2, dev, set[0])) return ZYFA_ERR_CUDA;
    e = launch_dependent(boxes4_kernel<DQK, DV, NS>, grid, threads + 32, smem, stream, a, maps);
  } else {
    if (!prepare(pieces4_kernel<DQK, DV, NS>, 2, dev, set[1])) return ZYFA_ERR_CUDA;
    e = launch_dependent(pieces4_kernel<DQK, DV, NS>, grid, threads + 32, smem, stream, a);
  }
  if (e != cudaSuccess) return ZYFA_ERR_CUDA;
  return a.whole ? ZYFA_OK : launch_join<DV>(a, nsm, dev, stream);
}

// By the query heads of a KV head: up to 8 are a warp's; more come in chunks of up to 16, two sets that share the widened codes and whose
// registers leave room for two blocks an SM instead of three (64 requests of 500 to 8000 tokens, 4 KV heads of 16: 45 us, in chunks of 8 49; of 64 channels, 31 and 59).
template <int DQK, int DV>
zyfa_status_t launch4(Args& a, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  return a.group <= 8 ? launch4_as<DQK, DV, 1>(a, nsm, dev, ws, stream) : launch4_as<DQK, DV, 2>(a, nsm, dev, ws, stream);
}

}  // namespace decode4
}  // namespace zyfa
