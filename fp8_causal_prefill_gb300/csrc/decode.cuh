// Attention of one new token per request over a paged key/value cache: device code.
//
// One pass over the keys with the running maximum m and sum l of the softmax (in units of log2):
//   x_j = a q.k_j,  m' = max(m, max_j x_j),  l' = l 2^(m-m') + sum_j 2^(x_j-m'),  O' = O 2^(m-m') + sum_j 2^(x_j-m') v_j
// and out = dv O / l, lse = ln2 (m + log2 l), with a = scale dq dk log2(e).  A row is empty (0 and -inf) if l is 0, not where it
// is not above 0: a NaN score, or one of +inf, makes NaN of l and of the row, as in the formula, however its request is split.
//
// Bound: the cache is read once (H_kv (D_qk + D_v) values per token) and a key costs 2 (D_qk + D_v) operations per
// query head, so with the usual 1 to 16 heads per KV head this is far below the tensor cores and HBM is the limit.
// The design keeps the loads running:
//
// * A block takes KV heads side by side: a tile is a run of tokens of several heads, whose rows are neighbours in memory,
//   and each compute warp takes one head, one run of 16 or 32 of the tokens and up to 8 of the query heads of it.  Warps
//   share nothing but the ring of tiles.
// * Products run with the keys (or the channels of V) as the 16 rows of mma.sync and the query heads as its 8
//   columns: S^T = K q^T, O^T = V^T P^T.  Few heads waste no second half of a tile, K and V fragments come
//   straight from ldmatrix, and the accumulators of a 128-channel head take 32 registers.  An e4m3 K multiplies an e4m3 q
//   as it is (m16n8k32, accumulated exactly to fp32); V is widened to fp16 in registers (exact) and multiplies P in
//   fp16 lifted by 2^15, so that the weights keep 11 bits.  A bf16 V multiplies P as a sum of two bf16 numbers, the second what the
//   first rounded off, so that they keep 16.  (With one, which keeps 8, 256 tokens came out 0.0020 off, relative, where the rounding of the
//   output alone gives 0.0016.)  The second product takes 0.4% of the time of 64 ragged requests with 4 query heads per KV head (46.3 to
//   46.5 us), 1.4% with 16 (65.4 to 66.3), 9% with 32 over one KV head (44.5 to 48.7).  The rest of an fp16 weight is not kept: it would
//   take 0.6% of 128 requests' time (180.5 to 181.7 us) and 9 to 12% with 8 and more query heads per KV head (44.9 to 49.1), for an error of
//   0.00165 instead of 0.00166.
// * Work is split over (request, key tile) evenly whatever the lengths: the tiles of all requests are numbered one after
//   the other, with a gap behind each request for what its end costs, and each group of blocks (one block per chunk of heads) takes an
//   equal run of the numbers.  A block finds its run from seq_lens on the device, so the host never needs the lengths.
// * A request that lies in one group's run is written directly; otherwise each group leaves (m, l, O) of its
//   part in the workspace and a second kernel joins the parts in group order.  Where the table has room for a few tiles only (at
//   most kLongest), a group is a request, and there is no second kernel.
// * The join is launched while the first kernel still runs and waits for it on the device (programmatic dependent
//   launch), which hides its launch.
//
// Two kernels differ in how tiles arrive.  boxes_kernel: pages whose size is a multiple of 8 tokens, by TMA; a warp of its
// own loads a block's tiles, one box for K and one for V per page.  (Compute warps that loaded for themselves spent 500 to
// 950 clocks per tile on it, as long as on the tile.)  rows_kernel: any page size and stride, by cp.async; each warp
// loads its own tiles row by row into a ring of its own.
//
// Measured on the GPU, in captured graphs, with the bytes of the caches over the time, against 6.78 TB/s of a copy: 128 requests of 513
// to 16384 tokens, 8 KV heads of 128 e4m3 channels and 32 query heads, 178 to 180 us (6.7 TB/s; 0.87 of the DRAM's cycles, the tensor
// cores busy for 0.19 of the time); 64 ragged requests in bf16 46.5 us (5.4 TB/s), 9 requests of 16 heads of 192/128 e4m3 channels
// 59 us (6.0 TB/s).  The rest is the start (lengths, then pages, then tiles: three trips to memory) and the join, 6 to 8 us
// together, which is also what a short context takes: 256 tokens 6 us, one request of 32768 tokens 18 us.  (The call of the 256 tokens, with
// nothing else to do, takes the host 8 to 10.)
// With 16 query heads per KV head a byte meets twice the arithmetic and widening V takes as long as its load: 4.2 TB/s
// in e4m3, 5.7 in bf16.  (ldmatrix transposes bytes, so widening is one conversion per two values; with pairs of bytes and a
// permutation before it, 48.4 us instead of 45.9.)  Two column groups that share the fragments of K and V take 168 registers a
// thread, and with a third fewer warps the same time (48.7 to 47.6 us, 32 heads 37 to 41): chunks of 8 heads have a warp each.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "paged.cuh"
#include "ptx.cuh"

namespace zyfa {
namespace decode {

constexpr int kMaxSms = 160;          // the workspace is sized for at most this many SMs ...
constexpr int kMaxWarpsPerSm = 16;    // ... of this many compute warps
constexpr int kMaxDevices = 64;
constexpr int kSmemPerBlock = 232448, kSmemPerSm = 233472;
constexpr long long kWaitClocks = 1ll << 31, kShortWaitClocks = 1ll << 22;  // bound of every wait, about a second; that of the self-test

struct DecodeArgs {
  const uint8_t* q;
  long long q_batch;  // bytes
  CacheView cache;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  __nv_bfloat16* out;
  float* lse;
  const float *q_desc, *k_desc, *v_desc;
  int* status;
  float scale_log2;
  int desc_per_head, desc_request;  // one value a KV head; values from a request to the next (0: all take the same)
  int max_len;  // max_pages * page_size
  int B, H, group;
  uint32_t page_magic;  // floor(t / page_size) = t * page_magic >> page_shift for t < 2^30
  int page_shift;
  long long wait_clocks;
  int stalled;  // self-test: nothing is loaded
  // schedule and workspace
  int whole;                    // a group is a request; no join
  int groups, units;            // `units` blocks (boxes_kernel) or warps (rows_kernel) make a group
  int chunks, chunk_heads;      // the query heads of a KV head are cut into chunks of at most chunk_heads
  int heads, chunk_warps, subs; // of a block: KV heads, chunks of each, token runs of a tile (warps = the product)
  int stages, tile_tokens;      // of a ring; tokens of a tile, subs * turns * keys of a warp's turn
  int turns;                    // of a warp at a tile
  int tile_log2;                // of tile_tokens, a power of two
  int q_bytes;                  // of a block's queries in shared memory
  int box_log2;                 // tokens of a TMA box, at most a tile's
  int joint_k, joint_v;         // rows of 64 (or 192) bytes lie in shared memory in 128-byte columns across heads
  unsigned* starts;  // [B + 1], for more than kFewJoin requests: number of each one's first tile, then the numbers of a run
  float2* ml;        // [groups][2][H]
  float* part;       // [groups][2][H][DV]
};

// ------------------------------------------------------------------------------------------------
// warp-level pieces

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Waits for a phase, for at most `clocks`; the whole warp gets the same answer.
__device__ __forceinline__ bool mbar_wait_bounded(uint32_t bar, uint32_t parity, long long clocks) {
  bool done = ptx::mbar_try_wait(bar, parity);
  if (!done) {
    const long long t0 = clock64();
    do done = ptx::mbar_try_wait(bar, parity);
    while (!done && clock64() - t0 < clocks);
  }
  return __all_sync(0xffffffffu, done);
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}
// Untiled bulk copy: both addresses 16-byte aligned, a multiple of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
               "r"(bar)
               : "memory");
}

// 16 bytes global -> shared; `bytes` 0 writes zeros without reading.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two 16 x 16 matrices of bytes, transposed: lane 4r + c gets bytes 4c .. 4c + 3 of columns r (r[0], r[2]) and r + 8 (r[1], r[3]).
__device__ __forceinline__ void ldsm2t_bytes(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
enum { kF16, kBf16, kE4m3 };
// D += A B for 16 rows, 8 columns and a contraction of 16 (16-bit operands) or 32 (e4m3).
template <int KIND>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
#define ZYFA_MMA(SHAPE_AND_TYPES)                                                                                       \
  asm("mma.sync.aligned." SHAPE_AND_TYPES " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                      \
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                                                                  \
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (KIND == kF16)
    ZYFA_MMA("m16n8k16.row.col.f32.f16.f16.f32");
  else if constexpr (KIND == kBf16)
    ZYFA_MMA("m16n8k16.row.col.f32.bf16.bf16.f32");
  else
    ZYFA_MMA("m16n8k32.row.col.f32.e4m3.e4m3.f32");
#undef ZYFA_MMA
}
// Two e4m3 codes (low half of `x`) as two fp16 values.
__device__ __forceinline__ uint32_t widen(uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t x) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Pairs of fp32 values in one instruction, each rounded as alone.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tadd.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
template <bool FP8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  if constexpr (FP8)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// What pack2 rounded off two values, rounded itself: together they keep 16 bits or more of each.
__device__ __forceinline__ uint32_t pack2_rest(float lo, float hi, uint32_t rounded) {
  return pack2<false>(lo - __uint_as_float(rounded << 16), hi - __uint_as_float(rounded & 0xffff0000u));
}

template <bool FP8, int DQK, int DV>
struct Tile {
  static constexpr int kEs = FP8 ? 1 : 2;
  static constexpr int kRowK = DQK * kEs, kRowV = DV * kEs;
  static constexpr int kKeyBytes = kRowK + kRowV;
  static constexpr int kKeys = kKeyBytes <= 128 ? 32 : 16;  // per stage: 4 to 10 KiB
  static constexpr int kTileBytes = kKeys * kKeyBytes;
  static constexpr uint32_t kFull = kKeys == 32 ? 0xffffffffu : 0xffffu;
};

// K or V rows of a run of tokens lie in shared memory as columns of CB bytes, each [tokens][CB] with the 16-byte pieces of a
// row exchanged as TMA's 128-byte (64-byte) swizzle does, so that the 8 rows that one ldmatrix phase reads lie in 8
// different bank groups.  CB = 128 where the rows are a multiple of that.  Rows of an odd number of 64-byte halves are columns of
// 64 bytes, or (`joint`), where heads follow one another without a gap, 128-byte columns that two heads share: TMA spends
// its time by rows of a box, and half as long ones reached 5.3 of 6.8 TB/s.
template <int ROW>
constexpr bool kWhole = ROW % 128 == 0;

// Where one lane's ldmatrix reads go: piece p (16 bytes, p even, plus the lane's own 0 or 1) of row 16 n + the lane's, of one
// head, is at ((tile + base[n]) ^ flip) + add for the 64-byte half that p lies in (relative to the first half's column).
template <int ROW, int KB>
struct Reader {
  static constexpr int kHalves = ROW / 64;
  uint32_t base[KB], column, add[kWhole<ROW> ? 1 : kHalves], flip[kWhole<ROW> ? 1 : kHalves];

  // tokens: of a box; head: within the box, of `heads`; row, hi: the lane's row of the first 16 and its piece of a pair
  __device__ __forceinline__ void set(int tokens_log2, int head, int heads, int first_row, int row, int hi, bool joint) {
    const int tokens = 1 << tokens_log2;
    const bool wide = kWhole<ROW> || joint;
    const int cb = wide ? 128 : 64;
    column = tokens * cb;
    const uint32_t first = head * kHalves / (wide ? 2 : 1) * column;
#pragma unroll
    for (int n = 0; n < KB; ++n) {
      const int r = first_row + n * 16 + row, box = r >> tokens_log2, in = r & (tokens - 1);
      base[n] = first + box * heads * tokens * ROW + in * cb + ((hi ^ (wide ? in & 7 : (in >> 1) & 3)) << 4);
    }
    if constexpr (!kWhole<ROW>) {
#pragma unroll
      for (int j = 0; j < kHalves; ++j) {
        const int half = head * kHalves + j;
        add[j] = (wide ? half >> 1 : half) * column - first;
        flip[j] = wide ? (half & 1) << 6 : 0;
      }
    }
  }
  __device__ __forceinline__ uint32_t at(uint32_t tile, int n, int p) const {
    const int j = p / 4;
    if constexpr (kWhole<ROW>)
      return ((tile + base[n]) ^ ((p % 8) << 4)) + (j / 2) * column;
    else
      return ((tile + base[n]) ^ (flip[j] | (p % 4) << 4)) + add[j];
  }
};

// Address of 16-byte piece p of row r in a lone head's run of `tokens` rows that is not joint.
template <int ROW>
__device__ __forceinline__ uint32_t place(int tokens, int r, int p) {
  constexpr int CB = kWhole<ROW> ? 128 : 64, PIECES = CB / 16;
  const int c = p / PIECES, q = p % PIECES;
  return static_cast<uint32_t>((c * tokens + r) * CB + ((q ^ (CB == 128 ? (r & 7) : ((r >> 1) & 3))) << 4));
}

// What the load side tells the compute side about a stage.
struct Header {
  int b, flags;
  int valid;       // tokens of the request in the tile
  uint32_t boxes;  // boxes_kernel: those whose page is in the cache; rows_kernel: such rows
};
// first and last tile of a request's part; the part is the whole request; it begins the request; not every key is valid; the run's last tile
enum : int { kFirst = 1, kLast = 2, kDirect = 4, kSlot1 = 8, kPartial = 16, kEnd = 32 };

__device__ __forceinline__ int length_of(const DecodeArgs& a, int b) { return max(0, min(a.seq_lens[b], a.max_len)); }

__device__ __forceinline__ void page_of(const DecodeArgs& a, int t, int* p, int* off) {
  *p = static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(t)) * a.page_magic) >> a.page_shift);
  *off = t - *p * a.cache.page_size;
}

// The order of a block of 16 keys in the products.  e4m3: byte e of the register that lane 4r + c gets of V is the key whose row
// lane 4c + e gave the address of, and its halves are keys 2c, 2c + 1 and 2c + 8, 2c + 9 of the contraction, whose weights come from those
// rows of the scores.  Rows 8 to 15 of the scores are keys 12 to 15, 8 to 11, so that neither K's reads nor V's meet rows of the same
// remainder by 8, which lie in the same banks.
template <bool FP8>
__device__ __forceinline__ int key_row(int r) {  // the key in row r of the scores
  return FP8 && r >= 8 ? r ^ 4 : r;
}
template <bool FP8>
__device__ __forceinline__ int value_row(int lane) {  // the key whose row of V a lane gives the address of
  const int c = lane >> 2 & 3, e = lane & 3;
  return FP8 ? key_row<true>(2 * c + (e & 1) + (e >> 1) * 8) : (lane >> 4) * 8 + (lane & 7);
}

// ------------------------------------------------------------------------------------------------
// the state of a compute warp: up to 8 query heads against its tiles

template <bool FP8, int DQK, int DV>
struct Rows {
  using T = Tile<FP8, DQK, DV>;
  static constexpr int KT = T::kKeys, KB = KT / 16;
  static constexpr int kKSteps = T::kRowK / 32, kMTiles = DV / 16;
  static constexpr int kScoreKind = FP8 ? kE4m3 : kBf16, kValueKind = FP8 ? kF16 : kBf16;
  static constexpr float kLift = FP8 ? 15.0f : 0.0f;  // e4m3: weights in fp16 up to 2^15, so that light ones keep their bits
  static constexpr float kNoKey = 3.402823466e38f;    // ref before the first key: lifts every score above its negative over the limit

  uint32_t qf[kKSteps][2];      // B fragments of the queries
  float o[kMTiles][4], m[2], l[2];  // this lane's two heads
  F2 ref;                           // kLift - m
  float scale, dv;

  // Begins a request's part: its queries from shared memory, `count` dense rows.
  __device__ __forceinline__ void begin(uint32_t queries, int count, float scale_, float dv_, int lane) {
    // rows behind the last head repeat it: their columns are computed and never written
    const uint32_t row = queries + min(lane & 7, count - 1) * T::kRowK + (lane >> 3) * 16;
#pragma unroll
    for (int i = 0; i < kKSteps; i += 2) {
      uint32_t x[4];
      ldsm4(row + i * 32, x);
      qf[i][0] = x[0];
      qf[i][1] = x[1];
      qf[i + 1][0] = x[2];
      qf[i + 1][1] = x[3];
    }
#pragma unroll
    for (int i = 0; i < kMTiles; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    m[0] = m[1] = -INFINITY;
    ref = {kNoKey, kNoKey};
    l[0] = l[1] = 0.0f;
    scale = scale_;
    dv = dv_;
  }

  // One tile of K at ks and V at vs.  FULL: all keys are valid; else mask: those that are, at least one, and clear() is called
  // since V rows of the others may hold anything.
  template <bool FULL, typename F>
  __device__ __forceinline__ void tile(uint32_t ks, uint32_t vs, const Reader<T::kRowK, KB>& kr, const Reader<T::kRowV, KB>& vr, uint32_t mask,
                                       int lane, F clear) {
    // S^T: rows are keys, columns heads; then scores in units of log2
    F2 x[KB][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kKSteps; ++i) {
        uint32_t r[4];
        ldsm4(kr.at(ks, kb, 2 * i), r);
        mma<kScoreKind>(c, r[0], r[1], r[2], r[3], qf[i][0], qf[i][1]);
      }
      x[kb][0] = mul2({c[0], c[1]}, {scale, scale});
      x[kb][1] = mul2({c[2], c[3]}, {scale, scale});
    }
    if constexpr (!FULL) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (!((mask >> (kb * 16 + key_row<FP8>(j * 8 + (lane >> 2)))) & 1)) x[kb][j] = {-INFINITY, -INFINITY};
      clear();
    }
    // The reference m moves only when a key exceeds it: log2 of a weight is then above the lift.  (Before a part's first key
    // with a score above -inf m is -inf, and the log2 weight of such a key huge.)
    F2 y[KB][2];
    float over = -INFINITY;
    auto weigh = [&]() {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          y[kb][j] = add2(x[kb][j], ref);
          over = fmaxf(over, fmaxf(y[kb][j].x, y[kb][j].y));
        }
    };
    weigh();
    if (__any_sync(0xffffffffu, over > kLift)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = m[e];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) t = e ? fmaxf(t, fmaxf(x[kb][0].y, x[kb][1].y)) : fmaxf(t, fmaxf(x[kb][0].x, x[kb][1].x));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        const bool none = t == -INFINITY;
        const float f = none ? 1.0f : exp2_approx(m[e] - t);
        m[e] = t;
        (e ? ref.y : ref.x) = none ? kNoKey : kLift - t;
        l[e] *= f;
#pragma unroll
        for (int i = 0; i < kMTiles; ++i) {
          o[i][e] *= f;
          o[i][e + 2] *= f;
        }
      }
      weigh();
    }
    // weights, transposed into the B operand (keys are now the contraction)
    uint32_t pf[KB][2], rest[KB][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const F2 w = {exp2_approx(y[kb][j].x), exp2_approx(y[kb][j].y)};
        const F2 sum = add2({l[0], l[1]}, w);
        l[0] = sum.x;
        l[1] = sum.y;
        const uint32_t rounded = pack2<FP8>(w.x, w.y);
        pf[kb][j] = transpose8x8(rounded);
        if constexpr (!FP8) rest[kb][j] = transpose8x8(pack2_rest(w.x, w.y, rounded));
      }
    // O^T += V^T P^T: rows are channels of V
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < kMTiles; i += 2) {
          // a register holds four keys of a channel, in the order of the contraction (see key_row)
          uint32_t r[4];
          ldsm2t_bytes(vr.at(vs, kb, i), r);
          mma<kValueKind>(o[i], widen(r[0]), widen(r[1]), widen_hi(r[0]), widen_hi(r[1]), pf[kb][0], pf[kb][1]);
          mma<kValueKind>(o[i + 1], widen(r[2]), widen(r[3]), widen_hi(r[2]), widen_hi(r[3]), pf[kb][0], pf[kb][1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kMTiles; ++i) {
          uint32_t r[4];
          ldsm4t(vr.at(vs, kb, 2 * i), r);
          mma<kValueKind>(o[i], r[0], r[1], r[2], r[3], pf[kb][0], pf[kb][1]);
          mma<kValueKind>(o[i], r[0], r[1], r[2], r[3], rest[kb][0], rest[kb][1]);
        }
      }
    }
  }

  // Ends a request's part: writes its rows (`count` query heads from `first`), or (m, l, O) to part `slot` of the workspace.
  __device__ __forceinline__ void finish(const DecodeArgs& a, int b, int first, int count, bool direct, long long slot, int lane) {
    const int t4 = lane & 3, g8 = lane >> 2;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float sum = total(e);
      const int head = t4 * 2 + e;
      if (head < count) {
        const long long row = (direct ? static_cast<long long>(b) : slot) * a.H + first + head;
        const float f = !direct ? dv : sum == 0.0f ? 0.0f : dv / sum;
        if (g8 == 0) put_sums(a, row, direct, m[e], sum);
        __nv_bfloat16* out = a.out + row * DV;
        float* part = a.part + row * DV;
        if (direct) {
#pragma unroll
          for (int i = 0; i < kMTiles; ++i) {
            const float y0 = o[i][e] * f, y1 = o[i][e + 2] * f;
            out[i * 16 + g8] = __float2bfloat16_rn(y0);
            out[i * 16 + g8 + 8] = __float2bfloat16_rn(y1);
          }
        } else {
          put_o(part, e, f, g8);
        }
      }
    }
  }

  // The same for a request's part whose tiles' token runs `subs` warps shared (this one the sub-th): they leave (m, l, O) in
  // shared memory, meet, join them in order, each warp some of the heads, and meet again before the memory is used anew.
  // all_ml, all_o: [subs][8] and [subs][8][DV], `stride` warps from one sub's to the next; meet() is false if it gave up.
  template <typename F>
  __device__ __forceinline__ bool finish_shared(const DecodeArgs& a, int b, int first, int count, bool direct, long long slot, int lane, int sub,
                                                int subs, int stride, float2* all_ml, float* all_o, F meet) {
    const int g8 = lane >> 2;
    float2* my_ml = all_ml + sub * stride * 8;
    float* my_o = all_o + sub * stride * 8 * DV;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float sum = total(e);
      const int head = (lane & 3) * 2 + e;
      if (g8 == 0) my_ml[head] = make_float2(m[e], sum);
      put_o(my_o + head * DV, e, dv, g8);
    }
    if (!meet()) return false;
    constexpr int V = DV / 32;
    for (int head = sub; head < count; head += subs) {
      float M = -INFINITY, L = 0.0f, x[V] = {};
      for (int k = 0; k < subs; ++k) M = fmaxf(M, all_ml[k * stride * 8 + head].x);
      for (int k = 0; k < subs; ++k) {
        const float2 ml = all_ml[k * stride * 8 + head];
        const float e = ml.x == -INFINITY ? 0.0f : exp2_approx(ml.x - M);  // 0 for a run without a valid key, whose O is 0
        L = fmaf(ml.y, e, L);
        const float* y = all_o + (k * stride * 8 + head) * DV + lane * V;
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
  __device__ __forceinline__ float total(int e) const {
    float sum = l[e];
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
  __device__ __forceinline__ void put_o(float* to, int e, float f, int g8) const {
#pragma unroll
    for (int i = 0; i < kMTiles; ++i) {
      to[i * 16 + g8] = o[i][e] * f;
      to[i * 16 + g8 + 8] = o[i][e + 2] * f;
    }
  }
};

// The Readers of a warp whose run of keys begins at row `first_row` of a tile of boxes.
template <bool FP8, int DQK, int DV, int KB>
__device__ __forceinline__ void set_readers(int lane, int tokens_log2, int head, int heads, int first_row, bool joint_k, bool joint_v,
                                            Reader<Tile<FP8, DQK, DV>::kRowK, KB>* k, Reader<Tile<FP8, DQK, DV>::kRowV, KB>* v) {
  k->set(tokens_log2, head, heads, first_row, key_row<FP8>(lane & 15), lane >> 4, joint_k);
  v->set(tokens_log2, head, heads, first_row, value_row<FP8>(lane), FP8 ? lane >> 4 : lane >> 3 & 1, joint_v);
}

// ------------------------------------------------------------------------------------------------
// the schedule

// The tiles (of a.tile_tokens tokens) of all requests are numbered one after the other, with a gap of kGap behind each request for what
// its end costs; a group's run is an equal piece of the numbers.  find() gives the request and the tile within it that run `g` begins
// with and the numbers from there to the run's end (0: the run has no tile), for every thread that asks (`finds`; of one
// warp, the same g).  Numbers fit 32 bits (the host has checked their sum).
//
// The gap keeps a run of many short requests from being the last to end: 53 requests of 10 to 35,000 tokens (one KV head, bf16) 22.2
// us without, 18.5 with a gap of 1, 18.1 with 2 (and 18.0 with 3); 42 requests with 14 query heads 30.0, 26.5, 25.4 (24.8).
constexpr unsigned kGap = 2;
// Up to kFew requests warps read all lengths themselves, else blocks do with barriers: 189 requests 20.0 us instead of 21.6.
constexpr int kFew = 256;
// The join reads them up to kFewJoin, else what the first kernel left (from the first request on 0.2 to 0.4 us more for short
// batches; 256 requests of 32 heads, 100 tokens each: 21.0 us instead of 23.2).
constexpr int kFewJoin = 128;  // four a lane

struct Schedule {
  unsigned total = 0, per = 0;  // numbers, and those of a run

  static __device__ __forceinline__ unsigned tiles_of(const DecodeArgs& a, int length) { return (length + a.tile_tokens - 1u) >> a.tile_log2; }
  static __device__ __forceinline__ unsigned tiles(const DecodeArgs& a, int b) { return b < a.B ? tiles_of(a, length_of(a, b)) : 0u; }
  static __device__ __forceinline__ unsigned numbers(unsigned tiles) { return tiles ? tiles + kGap : 0; }
  __device__ __forceinline__ void set(const DecodeArgs& a, unsigned sum) {
    total = sum ? sum - kGap : 0;
    per = (total + a.groups - 1) / a.groups;
  }

  // Up to 32 N requests: every warp by itself, N requests a lane, whose tiles n are, without a barrier.  Returns the lane's first number.
  template <int N>
  __device__ __forceinline__ unsigned scan_few(const DecodeArgs& a, const unsigned (&n)[N]) {
    const int lane = threadIdx.x & 31;
    unsigned sum = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += numbers(n[i]);
    unsigned incl = sum;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const unsigned o = __shfl_up_sync(0xffffffffu, incl, s);
      if (lane >= s) incl += o;
    }
    set(a, __shfl_sync(0xffffffffu, incl, 31));
    return incl - sum;
  }
  template <int N>
  __device__ __forceinline__ void find_few(const DecodeArgs& a, unsigned g, int* b, unsigned* tile, int* left) {
    unsigned n[N], at = 0, number = 0, rest = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = tiles(a, (threadIdx.x & 31) * N + i);
    unsigned start = scan_few<N>(a, n);
    const unsigned first = g * per;
    bool here = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {  // the first of this lane's requests that has a tile from number `first` on
      if (!here && n[i] && start + n[i] > first) {
        at = (threadIdx.x & 31) * N + i;
        number = max(start, first);
        rest = number - start;
        here = true;
      }
      if (N * 32 > kFewJoin && blockIdx.x == 0 && threadIdx.x < 32 && threadIdx.x * N + i < a.B) a.starts[threadIdx.x * N + i] = start;
      start += numbers(n[i]);
    }
    if (N * 32 > kFewJoin && blockIdx.x == 0 && threadIdx.x == 0) a.starts[a.B] = per;
    const unsigned hit = __ballot_sync(0xffffffffu, here);
    const int l = hit ? __ffs(hit) - 1 : 0;
    *b = static_cast<int>(__shfl_sync(0xffffffffu, at, l));
    *tile = __shfl_sync(0xffffffffu, rest, l);
    number = __shfl_sync(0xffffffffu, number, l);
    *left = hit ? max(0, static_cast<int>(min(first + per, total) - number)) : 0;
  }
  // Numbers of request b's first tile and, were it one longer, of its next, from this lane's N lengths (behind the last one: 0).
  template <int N>
  __device__ __forceinline__ void bounds_few(const DecodeArgs& a, const int (&lengths)[N], int b, unsigned* p0, unsigned* p1) {
    unsigned n[N], len = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n[i] = tiles_of(a, lengths[i]);
    unsigned mine = scan_few<N>(a, n);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < b % N) mine += numbers(n[i]);
      if (i == b % N) len = n[i];
    }
    *p0 = __shfl_sync(0xffffffffu, mine, b / N);
    *p1 = *p0 + __shfl_sync(0xffffffffu, len, b / N);
  }

  // Any number, the whole block: prefix: [blockDim.x] and sums: [warps] in shared memory.  Leaves a.starts for the join.
  __device__ __forceinline__ void find(const DecodeArgs& a, unsigned* prefix, unsigned* sums, bool finds, unsigned g, int* b,
                                       unsigned* tile, int* left) {
    // (code that a case does not need costs it: four requests a lane for all made short batches 0.2 us slower, eight 0.5)
    if (a.B <= 32) return find_few<1>(a, g, b, tile, left);
    if (a.B <= 128) return find_few<4>(a, g, b, tile, left);
    if (a.B <= kFew) return find_few<8>(a, g, b, tile, left);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_threads = blockDim.x, warps = n_threads >> 5;
    unsigned sum = 0;
    for (int r = tid; r < a.B; r += n_threads) sum += numbers(tiles(a, r));
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < warps; ++i) sum += sums[i];
    set(a, sum);
    __syncthreads();
    const unsigned first = g * per;
    unsigned before = 0;
    *b = -1;
    *tile = 0;
    *left = 0;
    for (int b0 = 0; b0 < a.B; b0 += n_threads) {
      const unsigned n = numbers(tiles(a, b0 + tid));
      unsigned incl = n;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const unsigned o = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += o;
      }
      if (lane == 31) sums[warp] = incl;
      __syncthreads();
      unsigned all = 0, mine = 0;
      for (int i = 0; i < warps; ++i) {
        if (i == warp) mine = all;
        all += sums[i];
      }
      const unsigned start = before + mine + incl - n;
      prefix[tid] = start;
      if (blockIdx.x == 0 && b0 + tid < a.B) a.starts[b0 + tid] = start;
      __syncthreads();
      if (finds && *b < 0 && first < total && first < before + all) {
        int lo = 0, hi = min(n_threads, a.B - b0);  // prefix[lo] <= first, and the last such: requests without tiles are passed
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (prefix[mid] <= first) lo = mid; else hi = mid;
        }
        *b = b0 + lo;
        *tile = first - prefix[lo];
        unsigned number = first;
        const unsigned own = tiles(a, *b);
        if (*tile >= own) {  // in the gap behind it: on to the next (there is one: the last request's gap is not counted)
          number += own + kGap - *tile;
          *tile = 0;
          do ++*b;
          while (*b + 1 < a.B && tiles(a, *b) == 0);
        }
        *left = max(0, static_cast<int>(min(first + per, total) - number));
      }
      before += all;
      __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) a.starts[a.B] = per;
  }
};

// Where the load side of a ring is: the next tile.
struct Cursor {
  int b, len, t, left;     // request, its length, first token of the next tile, numbers from there to the run's end
  bool first, from_start;  // the tile begins a part; the part begins its request
  __device__ __forceinline__ void start(const DecodeArgs& a, int b_, unsigned tile, int left_) {
    b = b_;
    t = static_cast<int>(tile) * a.tile_tokens;
    left = left_;
    len = length_of(a, b);
    first = true;
    from_start = t == 0;
  }
  __device__ __forceinline__ bool ends(int tokens) const { return t + tokens >= len; }  // this tile, its request
  __device__ __forceinline__ int left_after(int tokens) const { return left - 1 - (ends(tokens) ? static_cast<int>(kGap) : 0); }
  __device__ __forceinline__ int flags(int tokens) const {
    const bool end = ends(tokens), last = end || left == 1;
    return (first ? kFirst : 0) | (last ? kLast | (from_start && end ? kDirect : 0) | (from_start ? kSlot1 : 0) : 0) |
           (left_after(tokens) <= 0 ? kEnd : 0);
  }
  // to the next tile of the run, which has one
  __device__ __forceinline__ void advance(const DecodeArgs& a, int tokens) {
    first = false;
    t += tokens;
    if (t >= len) {
      do {
        ++b;
        len = length_of(a, b);
      } while (len == 0 && b + 1 < a.B);
      t = 0;
      first = true;
      from_start = true;
    }
  }
};

// ------------------------------------------------------------------------------------------------
// tiles by TMA

// Compute warps of a block at most.  Three blocks and their load warps share an SM: 15 warps of 128 registers a thread, or 9 of
// 168.  128 e4m3 requests, and 64 ragged ones in bf16: 179 and 46 us; two blocks of 8 (4) compute warps 187 and 48, two of 4 (2)
// 190 and 50, four of 2 191 and 47.
template <int KEY_BYTES>
constexpr int kBoxWarps = KEY_BYTES <= 320 ? 4 : 2;
// Tiles of a ring: the same 189 and 48 us with two, 179 and 46 with three, 187 and 49 with four.
constexpr int kMaxStages = 3, kMaxHeads = 8;
// A lone block takes 0.6 us a tile, the join 3 us.  With 4: 32 requests of 64 tokens (32 query heads, e4m3) 6.0 us instead of 7.9, one 5.5
// instead of 6.5, eight (16 heads, bf16) 5.7 instead of 7.0; with 8 also one of 128 tokens 8.1 instead of 6.8.  kLongest: 228
// requests (32 query and 8 KV heads, e4m3) of 128 tokens, 8 tiles, 14.8 us whole and 18.1 split, and with one such request among ones of one
// token 9.1 and 10.3; one of 256 tokens, 16 tiles, 13.2 whole and 10.2 split.  With no such bound, 228 requests of 1 to 16384 tokens took 598
// us instead of 127, since equal ones would have filled the GPU evenly.
constexpr int kSerial = 4, kLongest = 8;

template <bool FP8, int DQK, int DV>
__global__ void __launch_bounds__((kBoxWarps<Tile<FP8, DQK, DV>::kKeyBytes> + 1) * 32, 3)
    boxes_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using T = Tile<FP8, DQK, DV>;
  constexpr int KT = T::kKeys, KB = KT / 16, kMaxWarps = kBoxWarps<T::kKeyBytes> + 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ unsigned s_prefix[kMaxWarps * 32], s_sums[kMaxWarps];
  __shared__ __align__(16) Header s_header[kMaxStages];
  __shared__ float2 s_scale[kMaxStages][kMaxHeads];  // of the scores, and of V
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_meet[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x >> 5) - 1;  // compute warps; the next one loads
  const int S = a.stages, TT = a.tile_tokens;
  const uint32_t k_bytes = a.heads * TT * T::kRowK, stage_bytes = a.heads * TT * T::kKeyBytes;
  const uint32_t tiles_s = smem_addr(smem), query_s = tiles_s + S * stage_bytes, full_s = smem_addr(s_full), empty_s = smem_addr(s_empty);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full_s + 8 * i, 1);
      ptx::mbar_init(empty_s + 8 * i, warps);
    }
    for (int i = 0; i < a.heads * a.chunk_warps; ++i) ptx::mbar_init(smem_addr(s_meet + i), a.subs);
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (threadIdx.x == 32) {
    ptx::tma_prefetch_desc(&kmap);
    ptx::tma_prefetch_desc(&vmap);
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
    Cursor c;
    c.start(a, b, tile0, left);
    const int box = 1 << a.box_log2, row = lane << a.box_log2;  // this lane's box of a tile: its first token
    // the block's query rows: whole heads, or (more chunks than warps) part of one head's
    const int first_q = head0 * a.group + chunk0 * a.chunk_heads;
    const int queries = chunk_units > 1 ? min(a.chunk_warps * a.chunk_heads, a.group - chunk0 * a.chunk_heads)
                                   : min(a.heads, a.cache.H_kv - head0) * a.group;
    // The pages of 32 boxes of the request at a time (a tile's boxes are among one such 32), the next 32, or the first ones of
    // the next request, being read meanwhile; likewise (lane: a head) the next request's descales.
    auto pages = [&](int request, int len, int box0) {
      const int t = (box0 + lane) << a.box_log2;
      if (t >= len) return -1;
      int p, off;
      page_of(a, t, &p, &off);
      return a.table[request * a.table_stride + p];
    };
    struct Descales {
      float q, k, v;
    };
    auto descales = [&](int request) {
      Descales d = {1.0f, 1.0f, 1.0f};
      if (FP8 && lane < a.heads) {
        const int i = a.desc_per_head ? request * a.desc_request + min(head0 + lane, a.cache.H_kv - 1) : 0;
        if (a.q_desc) d.q = a.q_desc[i];
        if (a.k_desc) d.k = a.k_desc[i];
        if (a.v_desc) d.v = a.v_desc[i];
      }
      return d;
    };
    int next_b = 0, next_len = 0, pg_next = -1;
    int pg_now = pages(c.b, c.len, c.t >> a.box_log2 & ~31);
    Descales desc = descales(c.b), desc_next = desc;
    auto look_ahead = [&](bool new_request) {
      if (new_request) {
        next_len = 0;
        if (((c.len - c.t + TT - 1) >> a.tile_log2) + static_cast<int>(kGap) < c.left)  // the run goes on behind this request
          for (next_b = c.b + 1; next_b < a.B && next_len == 0; ++next_b) next_len = length_of(a, next_b);
        --next_b;
        if (next_len > 0) desc_next = descales(next_b);
      }
      const int box0 = (c.t >> a.box_log2 & ~31) + 32;
      pg_next = box0 << a.box_log2 < c.len ? pages(c.b, c.len, box0) : next_len > 0 ? pages(next_b, next_len, 0) : -1;
    };
    bool bad = false;
    int stage = 0;
    uint32_t parity = 1;  // a new barrier counts as one whose phase before its first has ended
    bool begun = false;
    while (true) {
      if (!mbar_wait_bounded(empty_s + 8 * stage, parity, a.wait_clocks)) {
        if (lane == 0) atomicOr(a.status, kStatusTimeoutBit);
        break;
      }
      const uint32_t ks = tiles_s + stage * stage_bytes, bar = full_s + 8 * stage;
      const int valid = min(TT, c.len - c.t);
      int p, off;
      page_of(a, c.t + row, &p, &off);
      const int pg = __shfl_sync(0xffffffffu, pg_now, (c.t >> a.box_log2 & 31) + lane);
      const bool ok = row < valid && pg >= 0 && pg < a.cache.num_pages;
      const unsigned boxes = __ballot_sync(0xffffffffu, ok);
      bad |= row < valid && !ok;
      // the copies first: the barrier's phase cannot end before the arrival below
      if (ok) {
        const uint32_t at = ks + lane * (a.heads * box) * T::kRowK, vt = ks + k_bytes + lane * (a.heads * box) * T::kRowV;
        const bool jk = !kWhole<T::kRowK> && a.joint_k, jv = !kWhole<T::kRowV> && a.joint_v;
        tma_load_5d(at, &kmap, bar, 0, off, jk ? head0 * T::kRowK / 128 : 0, jk ? 0 : head0, pg);
        tma_load_5d(vt, &vmap, bar, 0, off, jv ? head0 * T::kRowV / 128 : 0, jv ? 0 : head0, pg);
      }
      if (c.first && lane < a.heads) s_scale[stage][lane] = {a.scale_log2 * desc.q * desc.k, desc.v};
      __syncwarp();
      if (lane == 0) {
        const bool whole = valid == TT && boxes == 0xffffffffu >> (32 - (TT >> a.box_log2));
        s_header[stage] = {c.b, c.flags(TT) | (whole ? 0 : kPartial), valid, boxes};
        const uint32_t q_bytes = c.first ? queries * T::kRowK : 0;
        if (c.first) bulk_load(query_s + stage * a.q_bytes, a.q + c.b * a.q_batch + static_cast<long long>(first_q) * T::kRowK, q_bytes, bar);
        ptx::mbar_arrive_expect_tx(bar, (__popc(boxes) << a.box_log2) * a.heads * T::kKeyBytes + q_bytes);
      }
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
        pg_now = pg_next;
        desc = desc_next;
        look_ahead(true);
      } else if ((c.t >> a.box_log2 & 31) == 0) {
        pg_now = pg_next;
        look_ahead(false);
      }
      if (++stage == S) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (bad) atomicOr(a.status, kStatusBadPageBit);
    return;
  }

  Reader<T::kRowK, KB> kr;
  Reader<T::kRowV, KB> vr;
  const int run_keys = a.turns * KT;
  set_readers<FP8, DQK, DV, KB>(lane, a.box_log2, head, a.heads, sub * run_keys, a.joint_k, a.joint_v, &kr, &vr);
  // bytes from a box to the next, and from a row of one to the next
  const uint32_t k_box = a.heads * T::kRowK << a.box_log2, v_box = a.heads * T::kRowV << a.box_log2;
  const uint32_t k_pitch = kWhole<T::kRowK> || a.joint_k ? 128 : 64, v_pitch = kWhole<T::kRowV> || a.joint_v ? 128 : 64;
  const uint32_t my_query = query_s + (head * a.group + (chunk - chunk0) * a.chunk_heads) * T::kRowK;
  // where warps that share a head's tokens meet
  const int peers = a.heads * a.chunk_warps, peer = warp % peers;
  float2* all_ml = reinterpret_cast<float2*>(smem + S * (stage_bytes + a.q_bytes)) + peer * 8;
  float* all_o = reinterpret_cast<float*>(smem + S * (stage_bytes + a.q_bytes) + warps * 64) + peer * 8 * DV;
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
  Rows<FP8, DQK, DV> rows;
  int stage = 0;
  uint32_t parity = 0;
  while (true) {
    if (!mbar_wait_bounded(full_s + 8 * stage, parity, a.wait_clocks)) {
      give_up(stage, parity);
      return;
    }
    const Header h = s_header[stage];
    const uint32_t ks = tiles_s + stage * stage_bytes, vs = ks + k_bytes;
    if (!idle) {
      if (h.flags & kFirst) rows.begin(my_query + stage * a.q_bytes, nq, s_scale[stage][head].x, s_scale[stage][head].y, lane);
      for (int turn = 0; turn < a.turns; ++turn) {
        // (a warp's run of keys begins with a box, or lies in one)
        const int r = turn * KT, boxes = r >> a.box_log2, in = r & ((1 << a.box_log2) - 1);
        const uint32_t kt = ks + boxes * k_box + in * k_pitch, vt = vs + boxes * v_box + in * v_pitch;
        if (!(h.flags & kPartial)) {
          rows.template tile<true>(kt, vt, kr, vr, T::kFull, lane, []() {});
          continue;
        }
        const int row0 = sub * run_keys + r;
        if (h.valid <= row0) break;
        uint32_t mask = T::kFull >> (KT - min(KT, h.valid - row0));
        mask &= __ballot_sync(0xffffffffu, h.boxes >> ((row0 + lane) >> a.box_log2 & 31) & 1);
        if (mask)
          rows.template tile<false>(kt, vt, kr, vr, mask, lane, [&]() {
            // whatever V holds behind the request's end is not a number to multiply by 0: its pieces as this warp reads them
#pragma unroll
            for (int n = 0; n < KB; ++n) {
              const int row = value_row<FP8>(lane);
              if (!((mask >> (n * 16 + row)) & 1))
#pragma unroll
                for (int p = 0; p < T::kRowV / 16; p += 2) ptx::st_shared_v4(vr.at(vt, n, p), 0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();  // before a later TMA load into this stage
            __syncwarp();
          });
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
// tiles by cp.async, row by row: any page size, any stride

constexpr int kRowStages = 3;

template <int KEY_BYTES>
constexpr int kRowWarps = KEY_BYTES <= 320 ? 12 : 8;

template <bool FP8, int DQK, int DV>
__global__ void __launch_bounds__((kRowWarps<Tile<FP8, DQK, DV>::kKeyBytes>) * 32, 1) rows_kernel(const __grid_constant__ DecodeArgs a) {
  using T = Tile<FP8, DQK, DV>;
  constexpr int KT = T::kKeys, KB = KT / 16, kLog2 = KT == 32 ? 5 : 4, kMaxWarps = kRowWarps<T::kKeyBytes>, S = kRowStages;
  constexpr int kPiecesK = T::kRowK / 16, kPiecesV = T::kRowV / 16;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ unsigned s_prefix[kMaxWarps * 32], s_sums[kMaxWarps];
  __shared__ __align__(16) Header s_header[kMaxWarps][S];
  __shared__ float2 s_scale[kMaxWarps][S];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_predecessor();
  let_successor_start();
  const unsigned w = warp * gridDim.x + blockIdx.x, g = w / a.units;  // few workers are spread over the blocks
  Schedule plan;
  int b, left;
  unsigned tile0;
  plan.find(a, s_prefix, s_sums, g < static_cast<unsigned>(a.groups), g, &b, &tile0, &left);
  if (g >= static_cast<unsigned>(a.groups) || left == 0) return;
  const int unit = static_cast<int>(w % a.units), hk = unit / a.chunks, chunk = unit % a.chunks;
  const int q0 = hk * a.group + chunk * a.chunk_heads, nq = min(a.chunk_heads, a.group - chunk * a.chunk_heads);
  const uint8_t* kbase = a.cache.k + hk * a.cache.k_head;
  const uint8_t* vbase = a.cache.v + hk * a.cache.v_head;
  const uint32_t tiles_s = smem_addr(smem) + warp * S * T::kTileBytes;
  const uint32_t query_s = smem_addr(smem) + (blockDim.x >> 5) * S * T::kTileBytes + warp * S * a.q_bytes;

  Cursor c;
  c.start(a, b, tile0, left);
  int pg, off;  // page and offset in it of token c.t + lane
  bool bad = false;
  auto look_up = [&]() {
    pg = -1;
    off = 0;
    if (lane < KT && c.t + lane < c.len) {
      int p;
      page_of(a, c.t + lane, &p, &off);
      pg = a.table[c.b * a.table_stride + p];
    }
  };
  look_up();
  auto issue = [&](int stage) {
    if (c.left > 0) {
      const bool inside = lane < KT && c.t + lane < c.len, ok = inside && pg >= 0 && pg < a.cache.num_pages;
      bad |= inside && !ok;
      const unsigned mask = __ballot_sync(0xffffffffu, ok);
      const uint32_t ks = tiles_s + stage * T::kTileBytes, vs = ks + KT * T::kRowK;
      const long long krow = ok ? pg * a.cache.k_page + off * a.cache.k_tok : 0;
      const long long vrow = ok ? pg * a.cache.v_page + off * a.cache.v_tok : 0;
#pragma unroll
      for (int i = 0; i < KT * kPiecesK / 32; ++i) {
        const int x = i * 32 + lane, r = x / kPiecesK, p = x % kPiecesK;
        copy16(ks + place<T::kRowK>(KT, r, p), kbase + __shfl_sync(0xffffffffu, krow, r) + p * 16, (mask >> r) & 1 ? 16 : 0);
      }
#pragma unroll
      for (int i = 0; i < KT * kPiecesV / 32; ++i) {
        const int x = i * 32 + lane, r = x / kPiecesV, p = x % kPiecesV;
        copy16(vs + place<T::kRowV>(KT, r, p), vbase + __shfl_sync(0xffffffffu, vrow, r) + p * 16, (mask >> r) & 1 ? 16 : 0);
      }
      if (c.first) {
        const uint8_t* q = a.q + c.b * a.q_batch + static_cast<long long>(q0) * T::kRowK;
        for (int x = lane; x < nq * kPiecesK; x += 32) copy16(query_s + stage * a.q_bytes + x * 16, q + x * 16, 16);
      }
      if (lane == 0) {
        s_header[warp][stage] = {c.b, c.flags(KT), KT, mask};
        if (c.first) {
          float2 scale = {a.scale_log2, 1.0f};
          if (FP8) {
            const int di = a.desc_per_head ? c.b * a.desc_request + hk : 0;
            scale.x *= (a.q_desc ? a.q_desc[di] : 1.0f) * (a.k_desc ? a.k_desc[di] : 1.0f);
            scale.y = a.v_desc ? a.v_desc[di] : 1.0f;
          }
          s_scale[warp][stage] = scale;
        }
      }
      c.left = c.left_after(KT);
      if (c.left > 0) {
        c.advance(a, KT);
        look_up();
      }
    }
    copy_commit();
  };

  Reader<T::kRowK, KB> kr;
  Reader<T::kRowV, KB> vr;
  set_readers<FP8, DQK, DV, KB>(lane, kLog2, 0, 1, 0, false, false, &kr, &vr);
  Rows<FP8, DQK, DV> rows;
  for (int i = 0; i < S - 1; ++i) issue(i);
  int stage = 0;
  while (true) {
    copy_wait<S - 2>();
    __syncwarp();  // this tile has landed, and every lane has read the one before it, whose stage is refilled
    issue(stage == 0 ? S - 1 : stage - 1);
    const Header h = s_header[warp][stage];
    const uint32_t ks = tiles_s + stage * T::kTileBytes, vs = ks + KT * T::kRowK;
    if (h.flags & kFirst) rows.begin(query_s + stage * a.q_bytes, nq, s_scale[warp][stage].x, s_scale[warp][stage].y, lane);
    if (h.boxes == T::kFull)
      rows.template tile<true>(ks, vs, kr, vr, T::kFull, lane, []() {});
    else if (h.boxes)
      rows.template tile<false>(ks, vs, kr, vr, h.boxes, lane, []() {});  // rows that are not valid were filled with zeros
    if (h.flags & kLast) rows.finish(a, h.b, q0, nq, h.flags & kDirect, static_cast<long long>(g) * 2 + (h.flags & kSlot1 ? 1 : 0), lane);
    if (h.flags & kEnd) break;
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  copy_wait<0>();
  if (bad) atomicOr(a.status, kStatusBadPageBit);
}

// ------------------------------------------------------------------------------------------------
// the join

// Joins the parts of the requests that several groups worked on, and writes the rows of empty requests.  W warps take a (request,
// head): every W-th part each, 32 at a time.  A lane reads one part's maximum and sum while the rows of O come in, none of
// which depends on another; then the warps meet in shared memory in a fixed order.  A block takes ROWS of them (W = 1), or VEC
// * 32 of the channels of one.  Latency bounds it: 3 to 4 us after the first kernel's end.
// The blocks an SM leave registers for BATCH rows on their way; with 64 a thread the compiler read them one after the other (20.7 us
// instead of 18.0 for 32 rows of 228 parts).
template <int DV, int W, int ROWS, int VEC, int BATCH>
__global__ void __launch_bounds__(W * ROWS * 32, W == 16 ? 1 : W == 4 ? 7 : 3) join_kernel(const __grid_constant__ DecodeArgs a) {
  static_assert(W == 1 || ROWS == 1);
  constexpr int kThreads = W * 32, D = VEC * 32;
  struct alignas(VEC * 4) Vec {
    float y[VEC];
  };
  __shared__ float s_o[W][D], s_m[W], s_l[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d0 = blockIdx.y * D;
  // Up to kFewJoin requests the bounds come from their lengths, read before the first kernel has ended.  It does not write them; what
  // did had ended, and its writes were visible, when that kernel's blocks came from their own wait, after which each let this one
  // start.  Only this SM's L1 could still hold what was there before, and these loads pass it by; of more than 32 requests a block
  // makes them once.
  __shared__ __align__(16) int s_length[kFewJoin];
  auto early = [&](int i) { return i < a.B ? max(0, min(load_relaxed(a.seq_lens + i), a.max_len)) : 0; };
  if (a.B > 32 && a.B <= kFewJoin) {
    for (int i = threadIdx.x; i < kFewJoin; i += W * ROWS * 32) s_length[i] = early(i);
    __syncthreads();
  }
  const long long row = static_cast<long long>(blockIdx.x) * ROWS + (ROWS > 1 ? warp : 0);
  if (row >= static_cast<long long>(a.B) * a.H) return;
  const int b = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H), w = ROWS > 1 ? 0 : warp, tid = w * 32 + lane;
  Schedule plan;
  unsigned p0, p1;
  if (a.B <= 32) {
    const int n[1] = {early(lane)};
    plan.bounds_few<1>(a, n, b, &p0, &p1);
  } else if (a.B <= kFewJoin) {
    const int4 n = reinterpret_cast<const int4*>(s_length)[lane];
    plan.bounds_few<4>(a, {n.x, n.y, n.z, n.w}, b, &p0, &p1);
  }
  wait_for_predecessor();
  if (a.B > kFewJoin) {
    p0 = a.starts[b];
    p1 = p0 + Schedule::tiles(a, b);
    plan.per = a.starts[a.B];
  }
  const unsigned per = plan.per;
  if (p0 == p1) {
    for (int i = tid; i < D; i += kThreads) a.out[row * DV + d0 + i] = __float2bfloat16_rn(0.0f);
    if (a.lse && tid == 0 && d0 == 0) a.lse[row] = -INFINITY;
    return;
  }
  const int g0 = static_cast<int>(p0 / per), n = static_cast<int>((p1 - 1) / per) - g0 + 1;
  if (n == 1) return;
  // part i: group g0 + i, its slot 1 (a request that begins there) for the first, else slot 0
  auto part = [&](int i) { return (static_cast<long long>(g0 + i) * 2 + (i == 0 ? 1 : 0)) * a.H + h; };
  float m = -INFINITY, l = 0.0f, o[VEC] = {};
  for (int base = w; base < n; base += 32 * W) {
    const int count = min(32, (n - base + W - 1) / W);  // parts base, base + W, ...
    const float2 ml = lane < count ? a.ml[part(base + lane * W)] : make_float2(-INFINITY, 0.0f);
    float e = 0.0f;
    for (int k0 = 0; k0 < count; k0 += BATCH) {
      Vec x[BATCH];
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        if (k0 + k < count) x[k] = *reinterpret_cast<const Vec*>(a.part + part(base + (k0 + k) * W) * DV + d0 + lane * VEC);
      if (k0 == 0) {  // with the first rows on their way
        float top = ml.x;
#pragma unroll
        for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.0f : mn, f = exp2_approx(m - ref);
        e = exp2_approx(ml.x - ref);  // 0 for parts without a valid key
        m = mn;
        l = l * f + ml.y * e;  // this lane's share
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] *= f;
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const float ek = __shfl_sync(0xffffffffu, e, (k0 + k) & 31);
        if (k0 + k < count) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) o[j] = fmaf(x[k].y[j], ek, o[j]);
        }
      }
    }
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  if constexpr (W == 1) {
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    __nv_bfloat16* out = a.out + row * DV + d0 + lane * VEC;
#pragma unroll
    for (int j = 0; j < VEC; j += 2) *reinterpret_cast<__nv_bfloat162*>(out + j) = __floats2bfloat162_rn(o[j] * f, o[j + 1] * f);
    if (a.lse && lane == 0 && d0 == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) s_o[w][lane * VEC + j] = o[j];
    if (lane == 0) {
      s_m[w] = m;
      s_l[w] = l;
    }
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < W; ++i) M = fmaxf(M, s_m[i]);
    float e[W], L = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      e[i] = s_m[i] == -INFINITY ? 0.0f : exp2_approx(s_m[i] - M);
      L = fmaf(s_l[i], e[i], L);
    }
    for (int i = tid; i < D; i += kThreads) {
      float x = 0.0f;
#pragma unroll
      for (int j = 0; j < W; ++j) x = fmaf(s_o[j][i], e[j], x);
      a.out[row * DV + d0 + i] = __float2bfloat16_rn(L == 0.0f ? 0.0f : x / L);
    }
    if (a.lse && tid == 0 && d0 == 0) a.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
  }
}

// ------------------------------------------------------------------------------------------------
// host side

inline long long round_up(long long x, long long n) { return (x + n - 1) / n * n; }

// Parts that one request and head can have at most, for the workspace: one per group.  A group has at least H_kv warps per chunk
// of 8 query heads, and there are no more groups than tiles.
inline long long parts_at_most(int B, int H, int H_kv, long long max_len) {
  const long long warps = static_cast<long long>(H_kv) * ((H / H_kv + 7) / 8);
  return std::max(1ll, std::min(kMaxSms * kMaxWarpsPerSm / warps, B * ((max_len + 15) / 16)));
}

inline long long tiles_at_most(int B, long long max_len, int keys) { return B * ((max_len + keys - 1) / keys); }

// Boxes of `tokens` rows of `heads` heads of one page.  The column dimension follows the tokens, so that a box lands as
// [head][column][token][CB]; `joint`: the heads' rows as one, in columns of 128 bytes.
inline bool make_map(CUtensorMap* m, const uint8_t* base, bool fp8, int row, const CacheView& c, long long page, long long tok, long long head,
                     int tokens, int heads, bool joint) {
  const int es = fp8 ? 1 : 2, cb = row % 128 == 0 || joint ? 128 : 64;
  using u64 = cuuint64_t;
  using u32 = cuuint32_t;
  const u64 dims[5] = {u64(cb / es), u64(c.page_size), u64(joint ? static_cast<long long>(c.H_kv) * row / cb : row / cb), u64(joint ? 1 : c.H_kv),
                       u64(c.num_pages)};
  const u64 strides[4] = {u64(tok), u64(cb), u64(joint ? tok : head), u64(page)};
  const u32 box[5] = {u32(cb / es), u32(tokens), u32(joint ? heads * row / cb : row / cb), u32(joint ? 1 : heads), 1};
  const u32 estr[5] = {1, 1, 1, 1, 1};
  return encode_tensor_map(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint8_t*>(base), dims, strides, box,
                           estr, cb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Both kernels ask for the largest share of shared memory: an SM changes the share only when it is empty, so blocks
// launched beside a predecessor of another share would find too little (1.5 times the time, 128 requests).
template <typename K>
bool prepare(K* kernel, int smem, int dev, std::atomic<int>* set) {
  if (set[dev].load(std::memory_order_acquire) >= smem) return true;
  const void* f = reinterpret_cast<const void*>(kernel);
  if (cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess) return false;
  if (smem > 1 && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerBlock - 8192) != cudaSuccess) return false;
  set[dev].store(smem > 1 ? kSmemPerBlock : 1, std::memory_order_release);
  return true;
}

inline int log2_of(int power) {
  int n = 0;
  while ((1 << n) < power) ++n;
  return n;
}

// Fewest equal pieces of `n` that are at most `most`, as the size of a piece.
inline int piece(int n, int most) { return (n + (n + most - 1) / most - 1) / ((n + most - 1) / most); }

// Chunks of up to 8 query heads, as equal as they come.
inline void set_chunks(DecodeArgs& a) {
  a.chunks = (a.group + 7) / 8;
  a.chunk_heads = (a.group + a.chunks - 1) / a.chunks;
}

// A block of boxes_kernel: chunks of a head first (they read the same tile), then heads side by side, then runs of tokens.  False if
// this cache is for rows_kernel.  Shared memory: what a stage takes, and the warps' meeting.
template <bool FP8, int DQK, int DV>
bool plan_boxes(DecodeArgs& a, int nsm, int* stage_bytes, int* meeting_bytes) {
  using T = Tile<FP8, DQK, DV>;
  const CacheView& c = a.cache;
  constexpr int kWarps = kBoxWarps<T::kKeyBytes>;
  a.chunk_warps = piece(a.chunks, kWarps);
  a.heads = piece(c.H_kv, kWarps / a.chunk_warps);
  a.subs = 1;
  while (a.subs * 2 * a.heads * a.chunk_warps <= kWarps) a.subs *= 2;
  // Where chunks of one head share a tile it has fewer rows; as many more tokens keep its bytes, which the work per tile of
  // the load warp and of the barriers is spread over.
  a.turns = 1;
  while (a.turns * 2 * a.subs * a.heads <= kWarps) a.turns *= 2;
  a.tile_tokens = a.subs * a.turns * T::kKeys;
  a.units = (c.H_kv + a.heads - 1) / a.heads * ((a.chunks + a.chunk_warps - 1) / a.chunk_warps);
  // Boxes: as many tokens of a page as divide both the page and the tile.  A broadcast (stride 0) or very large stride has no
  // tensor map, and a page of an odd size no boxes that fill the swizzle pattern (8 rows).
  a.tile_log2 = log2_of(a.tile_tokens);
  int tokens = a.tile_tokens;
  while (tokens > 1 && c.page_size % tokens != 0) tokens /= 2;
  if (tokens < 8) return false;
  for (long long s : {c.k_page, c.k_tok, c.k_head, c.v_page, c.v_tok, c.v_head})
    if (s <= 0 || s >= (1ll << 40)) return false;
  a.box_log2 = log2_of(tokens);
  auto joint = [&](int row, long long head) {
    return row % 128 != 0 && head == row && static_cast<long long>(c.H_kv) * row % 128 == 0 && a.heads * row % 128 == 0;
  };
  a.joint_k = joint(T::kRowK, c.k_head);
  a.joint_v = joint(T::kRowV, c.v_head);
  // a block's queries: whole heads, or (more chunks than warps) part of one head's
  const int nq = a.chunks > a.chunk_warps ? a.chunk_warps * a.chunk_heads : a.heads * a.group;
  a.q_bytes = static_cast<int>(round_up(nq * T::kRowK, 16));
  const int warps = a.heads * a.chunk_warps * a.subs, stage = a.heads * a.tile_tokens * T::kKeyBytes + a.q_bytes;
  const int meeting = a.subs > 1 ? warps * 8 * (DV + 2) * 4 : 0;  // (m, l, O) of the warps that share a head's tokens
  // three blocks an SM, or fewer if they would not have two stages each
  constexpr int kStatic = 4096;  // the schedule's tables and headers, with the 1 KiB that each block takes
  int blocks = 3;
  while (blocks > 1 && blocks * (2 * stage + meeting + kStatic) > kSmemPerSm) --blocks;
  a.stages = std::min(kMaxStages, (std::min(kSmemPerSm / blocks - kStatic, kSmemPerBlock - 8192) - meeting) / stage);
  if (a.stages < 2) return false;
  // Runs that are equal whatever the lengths, and a join; or a request a group, and no join.  What that can cost is the tiles of the
  // longest request that the table has room for, which one block takes alone, be the others as short as they may: kLongest of them at
  // most; and of the tables that short, those whose blocks are at most kSerial tiles behind the equal split when all requests are as long.
  const long long most = std::max(1ll, (a.max_len + a.tile_tokens - 1ll) / a.tile_tokens), at_once = std::max(1ll, static_cast<long long>(nsm) * blocks / a.units);
  const long long turns_whole = (a.B + at_once - 1) / at_once * most, turns_split = (a.B * most + at_once - 1) / at_once;
  a.whole = most <= kLongest && turns_whole - turns_split <= kSerial;
  a.groups = static_cast<int>(a.whole ? a.B : std::min(at_once, a.B * most));
  *stage_bytes = stage;
  *meeting_bytes = meeting;
  return true;
}

template <bool FP8, int DQK, int DV>
cudaError_t launch_boxes(DecodeArgs& a, bool* done, int nsm, int dev, cudaStream_t stream) {
  using T = Tile<FP8, DQK, DV>;
  const CacheView& c = a.cache;
  CUtensorMap kmap, vmap;
  int stage, meeting;
  *done = plan_boxes<FP8, DQK, DV>(a, nsm, &stage, &meeting) &&
          make_map(&kmap, c.k, FP8, T::kRowK, c, c.k_page, c.k_tok, c.k_head, 1 << a.box_log2, a.heads, a.joint_k) &&
          make_map(&vmap, c.v, FP8, T::kRowV, c, c.v_page, c.v_tok, c.v_head, 1 << a.box_log2, a.heads, a.joint_v);
  if (!*done) {
    a.whole = 0;
    return cudaSuccess;
  }
  static std::atomic<int> set[kMaxDevices];
  if (!prepare(boxes_kernel<FP8, DQK, DV>, 2, dev, set)) return cudaErrorUnknown;
  return launch_dependent(boxes_kernel<FP8, DQK, DV>, dim3(static_cast<unsigned>(a.groups) * a.units), (a.heads * a.chunk_warps * a.subs + 1) * 32,
                          a.stages * stage + meeting, stream, a, kmap, vmap);
}

// Kernels that launch() enqueues (if the driver takes the tensor maps).
template <bool FP8, int DQK, int DV>
int launches(DecodeArgs& a, int nsm) {
  int stage, meeting;
  set_chunks(a);
  return plan_boxes<FP8, DQK, DV>(a, nsm, &stage, &meeting) && a.whole ? 1 : 2;
}

template <bool FP8, int DQK, int DV>
cudaError_t launch_rows(DecodeArgs& a, int nsm, int dev, cudaStream_t stream) {
  using T = Tile<FP8, DQK, DV>;
  a.subs = 1;
  a.tile_tokens = T::kKeys;
  a.tile_log2 = log2_of(T::kKeys);
  a.units = a.cache.H_kv * a.chunks;
  a.q_bytes = a.chunk_heads * T::kRowK;
  const int ring = kRowStages * (T::kTileBytes + a.q_bytes), most = std::min(kRowWarps<T::kKeyBytes>, (kSmemPerBlock - 8192) / ring);
  const long long resident = static_cast<long long>(nsm) * most;
  a.groups = static_cast<int>(std::max(1ll, std::min(resident / a.units, tiles_at_most(a.B, a.max_len, T::kKeys))));
  const long long w = static_cast<long long>(a.groups) * a.units;
  const unsigned grid = static_cast<unsigned>(w <= resident ? std::min<long long>(nsm, w) : (w + most - 1) / most);
  const int warps = static_cast<int>((w + grid - 1) / grid);
  static std::atomic<int> set[kMaxDevices];
  if (!prepare(rows_kernel<FP8, DQK, DV>, 2, dev, set)) return cudaErrorUnknown;
  return launch_dependent(rows_kernel<FP8, DQK, DV>, dim3(grid), warps * 32, ring * warps, stream, a);
}

template <bool FP8, int DQK, int DV>
zyfa_status_t launch(DecodeArgs& a, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  // workspace: plan, (m, l), O
  const long long parts = parts_at_most(a.B, a.H, a.cache.H_kv, a.max_len);
  a.starts = reinterpret_cast<unsigned*>(ws);
  ws += round_up((a.B + 2ll) * 4, 256);
  a.ml = reinterpret_cast<float2*>(ws);
  ws += round_up(2 * parts * a.H * 8, 256);
  a.part = reinterpret_cast<float*>(ws);
  set_chunks(a);
  bool done;
  cudaError_t e = launch_boxes<FP8, DQK, DV>(a, &done, nsm, dev, stream);
  if (e == cudaSuccess && !done) e = launch_rows<FP8, DQK, DV>(a, nsm, dev, stream);
  if (e != cudaSuccess) return ZYFA_ERR_CUDA;
  if (a.whole) return ZYFA_OK;
  // Few rows have many parts each; a ragged batch may have most of its parts in a few rows, whatever their average.  So a row has as
  // many warps as the GPU holds at once (53 ragged requests of 8 heads: 25.5 us with one, 22.2 with four; 6 requests of 12 heads
  // 20.6 with four, 17.4 with 16; 5 of 64 heads 11.9 with four, 10.8 with eight; 32 rows 19.3 with whole rows, 18.0 with their channels spread), and of many rows, most of
  // which lie in one or two groups, a warp takes one (32 short requests of 32 heads: 7.5 us, with four warps 8.4).
  const unsigned rows = static_cast<unsigned>(a.B) * a.H, sms = static_cast<unsigned>(nsm);
  const long long parts_each = a.groups / a.B;
  constexpr int V = DV / 32;
  static std::atomic<int> set[5][kMaxDevices];
  if (rows * V <= sms) {
    if (!prepare(join_kernel<DV, 16, 1, 1, 16>, 1, dev, set[0])) return ZYFA_ERR_CUDA;
    e = launch_dependent(join_kernel<DV, 16, 1, 1, 16>, dim3(rows, V), 512, 0, stream, a);
  } else if (rows <= sms) {
    if (!prepare(join_kernel<DV, 16, 1, V, 8>, 1, dev, set[1])) return ZYFA_ERR_CUDA;
    e = launch_dependent(join_kernel<DV, 16, 1, V, 8>, dim3(rows), 512, 0, stream, a);
  } else if (rows <= 3 * sms && parts_each > 8) {
    if (!prepare(join_kernel<DV, 8, 1, V, 8>, 1, dev, set[4])) return ZYFA_ERR_CUDA;
    e = launch_dependent(join_kernel<DV, 8, 1, V, 8>, dim3(rows), 256, 0, stream, a);
  } else if (rows <= 4 * sms || (rows <= 8 * sms && parts_each > 4) || parts_each > 8) {
    if (!prepare(join_kernel<DV, 4, 1, V, 8>, 1, dev, set[2])) return ZYFA_ERR_CUDA;
    e = launch_dependent(join_kernel<DV, 4, 1, V, 8>, dim3(rows), 128, 0, stream, a);
  } else {
    if (!prepare(join_kernel<DV, 1, 8, V, 8>, 1, dev, set[3])) return ZYFA_ERR_CUDA;
    e = launch_dependent(join_kernel<DV, 1, 8, V, 8>, dim3((rows + 7) / 8), 256, 0, stream, a);
  }
  return e == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}

}  // namespace decode

// Instantiated in zyfa_decode_fp8.cu and zyfa_decode_bf16.cu.
zyfa_status_t decode_fp8(decode::DecodeArgs& a, int D_qk, int nsm, int dev, uint8_t* ws, cudaStream_t stream);
zyfa_status_t decode_bf16(decode::DecodeArgs& a, int D_qk, int nsm, int dev, uint8_t* ws, cudaStream_t stream);
int decode_launches_fp8(decode::DecodeArgs& a, int D_qk, int nsm);
int decode_launches_bf16(decode::DecodeArgs& a, int D_qk, int nsm);

}  // namespace zyfa
