// Attention of one new token per request over a paged key/value cache.
//
// One pass over the keys with the running maximum m and sum l of the softmax (in units of log2):
//   x_j = a q.k_j,  m' = max(m, max_j x_j),  l' = l 2^(m-m') + sum_j 2^(x_j-m'),  O' = O 2^(m-m') + sum_j 2^(x_j-m') v_j
// and out = dv O / l, lse = ln2 (m + log2 l), with a = scale dq dk log2(e).
//
// Bound: the cache is read once (H_kv (D_qk + D_v) values per token) and a key costs 2 (D_qk + D_v) operations per
// query head, so with the usual 1 to 16 heads per KV head this is far below the tensor cores and HBM is the limit.
// The design keeps the loads running:
//
// * The unit of work is a warp.  It streams its own tiles of KT keys through a private ring of stages and shares
//   nothing with other warps, so nothing in the loop waits for another warp.  Tiles of pages whose size is a
//   multiple of 8 tokens arrive by TMA (one lane issues a box per page, K and V), others by cp.async row by row.
// * Products run with the keys (or the channels of V) as the 16 rows of mma.sync and the query heads as its 8
//   columns: S^T = K q^T, O^T = V^T P^T.  Groups of up to 8 heads waste no second half, K and V fragments come
//   straight from ldmatrix, and the accumulators of a 128-channel head take 32 registers.  An e4m3 K multiplies an e4m3 q
//   as it is (m16n8k32); V is widened to fp16 in registers (exact) and multiplies P in fp16 lifted by 2^15, so that the
//   weights keep 11 bits.
// * Work is split over (request, key tile) evenly whatever the lengths: the tiles of all requests are numbered one after
//   the other and each group of warps (one warp per KV head and chunk of 16 query heads) takes an equal run
//   of them.  A group finds its run from seq_lens on the device, so the host never needs the lengths.  Heads of one
//   group read the same tokens at the same time, whose rows are neighbours in memory.
// * A request that lies in one group's run is written directly; otherwise each group leaves (m, l, O) of its
//   part in the workspace and a second kernel joins the parts in group order.
// * Both kernels are launched while their predecessor on the stream still runs and wait for it on the device
//   (programmatic dependent launch), which hides their launches.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <utility>

#include "paged.cuh"
#include "ptx.cuh"

namespace {

constexpr int kWarps = 2;             // warps of a block; they never synchronise with one another
constexpr int kMaxSms = 160;          // the workspace is sized for at most this many SMs ...
constexpr int kMaxWarpsPerSm = 16;    // ... of this many warps
constexpr long long kWaitClocks = 1ll << 31;  // bound of every wait, about a second

struct DecodeArgs {
  const uint8_t* q;
  long long q_batch;  // bytes
  zyfa::CacheView cache;
  const int* table;
  long long table_stride;
  const int* seq_lens;
  __nv_bfloat16* out;
  float* lse;
  const float *q_desc, *k_desc, *v_desc;
  int* status;
  float scale_log2;
  int desc_per_head;
  int max_len;  // max_pages * page_size
  int B, H, group;
  uint32_t page_magic;  // floor(t / page_size) = t * page_magic >> page_shift for t < 2^30
  int page_shift;
  // schedule and workspace
  int groups, chunks, chunk_heads, units;  // units = H_kv * chunks warps make a group
  int q_bytes;                      // of a query slot in shared memory
  int box_tokens_log2, box_chunks;  // TMA boxes: tokens and 64- or 128-byte column chunks of one
  unsigned* starts;  // [B + 2]: first tile of each request, then the total, then the tiles per group
  float2* ml;    // [groups][2][H]
  float* part;   // [groups][2][H][DV]
};

// ------------------------------------------------------------------------------------------------
// warp-level pieces

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

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
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
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

template <bool FP8, int DQK, int DV>
struct Tile {
  static constexpr int kEs = FP8 ? 1 : 2;
  static constexpr int kRowK = DQK * kEs, kRowV = DV * kEs;
  static constexpr int kKeyBytes = kRowK + kRowV;
  // Keys per stage, stages per warp and most blocks per SM (registers): a stage is 4 to 10 KiB, and the warps of an
  // SM together keep 100 KiB or more in flight.
  static constexpr int kKeys = FP8 ? 32 : 16;
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kKeys * kKeyBytes;
  static constexpr int kHeaders = 128;  // headers and barriers of the stages
  static constexpr int blocks(int nt) { return kKeyBytes <= 128 ? (nt == 1 ? 8 : 6) : kTileBytes <= 4096 ? (nt == 1 ? 8 : 6) : nt == 1 ? 5 : 4; }
  static_assert(kStages * (32 + 8) <= kHeaders);
};

// A K or V tile lies in shared memory as column chunks of CB = 128 bytes (64 where rows are not a multiple of that), each
// [keys][CB] with the 16-byte pieces of a row exchanged as TMA's 128-byte (64-byte) swizzle does, so that the 8 rows
// one ldmatrix phase reads lie in 8 different bank groups.
template <int ROW>
constexpr int kChunkBytes = ROW % 128 == 0 ? 128 : 64;

// Address of 16-byte piece p of row r within a tile.  For a lane that reads pieces 2 i + hi (hi 0 or 1) of rows r + 16 n it is
// (lane_part(r, hi) ^ (2 i % pieces of CB) * 16) + constants, whatever the multiple of 1024 that the tile begins at.
template <int ROW, int KEYS>
__device__ __forceinline__ uint32_t place(int r, int p) {
  constexpr int CB = kChunkBytes<ROW>, PIECES = CB / 16;
  const int c = p / PIECES, q = p % PIECES;
  const int s = CB == 128 ? (r & 7) : ((r >> 1) & 3);
  return static_cast<uint32_t>((c * KEYS + r) * CB + ((q ^ s) << 4));
}

template <int ROW>
__device__ __forceinline__ uint32_t lane_part(int r, int hi) {
  constexpr int CB = kChunkBytes<ROW>;
  return static_cast<uint32_t>(r * CB + ((hi ^ (CB == 128 ? (r & 7) : ((r >> 1) & 3))) << 4));
}
template <int ROW, int KEYS>
__device__ __forceinline__ uint32_t lane_place(uint32_t base, int p, int row16) {  // base: the tile's start + lane_part; p even
  constexpr int CB = kChunkBytes<ROW>, PIECES = CB / 16;
  return (base ^ ((p % PIECES) << 4)) + ((p / PIECES) * KEYS + row16 * 16) * CB;
}

// What the load side tells the compute side about a stage.
struct Header {
  uint32_t mask;   // valid keys
  int b;
  int flags;
  int q_slot;
  float dq, dk, dv;
  int pad;
};
enum : int { kFirst = 1, kLast = 2, kDirect = 4, kSlot1 = 8 };

// Tiles of request b.
template <int KT>
__device__ __forceinline__ unsigned tiles_of(const DecodeArgs& a, int b) {
  return (max(0, min(__ldg(a.seq_lens + b), a.max_len)) + KT - 1u) / KT;
}

template <bool FP8, int DQK, int DV, int NT, bool TMA>
__global__ void __launch_bounds__(kWarps * 32, (Tile<FP8, DQK, DV>::blocks(NT)))
    decode_kernel(const __grid_constant__ DecodeArgs a, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
  using T = Tile<FP8, DQK, DV>;
  namespace ptx = zyfa::ptx;
  constexpr int KT = T::kKeys, KB = KT / 16;
  constexpr int kChunksK = T::kRowK / 16, kChunksV = T::kRowV / 16;  // 16-byte pieces of a row
  constexpr int kKSteps = T::kRowK / 32, kMTiles = DV / 16;
  constexpr int kScoreKind = FP8 ? kE4m3 : kBf16, kValueKind = FP8 ? kF16 : kBf16;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_for_predecessor();
  let_successor_start();

  // ---- this group's run of tiles (all counts fit 32 bits: the host has checked their sum)
  unsigned total = 0;
  for (int b = lane; b < a.B; b += 32) total += tiles_of<KT>(a, b);
  total = __reduce_add_sync(0xffffffffu, total);
  const unsigned w = blockIdx.x * kWarps + warp, g = w / a.units, unit = w % a.units;
  const unsigned per = (total + a.groups - 1) / a.groups, first = g * per;
  const bool works = g < static_cast<unsigned>(a.groups) && first < total, writes_plan = w == 0;
  if (!works && !writes_plan) return;
  int b = -1;
  unsigned tile0 = 0;  // tile of request b that the run begins with
  {
    unsigned before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const unsigned n = b0 + lane < a.B ? tiles_of<KT>(a, b0 + lane) : 0;
      const unsigned sum = __reduce_add_sync(0xffffffffu, n);
      if (writes_plan || first < before + sum) {
        unsigned incl = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const unsigned o = __shfl_up_sync(0xffffffffu, incl, s);
          if (lane >= s) incl += o;
        }
        if (writes_plan && b0 + lane < a.B) a.starts[b0 + lane] = before + incl - n;
        const unsigned hit = __ballot_sync(0xffffffffu, first < before + incl);
        if (hit && b < 0) {
          b = b0 + __ffs(hit) - 1;
          tile0 = first - __shfl_sync(0xffffffffu, before + incl - n, __ffs(hit) - 1);
          if (!writes_plan) break;
        }
      }
      before += sum;
    }
    if (writes_plan && lane == 0) {
      a.starts[a.B] = total;
      a.starts[a.B + 1] = per;
    }
    if (!works || b < 0) return;
  }
  const unsigned left = min(per, total - first);

  const int hk = static_cast<int>(unit) / a.chunks, chunk = static_cast<int>(unit) % a.chunks;
  const int h0 = hk * a.group + chunk * a.chunk_heads;                     // first query head of this warp
  const int nh = min(a.chunk_heads, a.group - chunk * a.chunk_heads);      // and how many
  const uint8_t* kbase = a.cache.k + hk * a.cache.k_head;
  const uint8_t* vbase = a.cache.v + hk * a.cache.v_head;
  // the warps' stages of K and V rows, then for each warp its headers and barriers and its query slots (one fewer than
  // stages: see the loop)
  uint8_t* mine = smem + kWarps * T::kStages * T::kTileBytes + warp * (T::kHeaders + (T::kStages - 1) * a.q_bytes);
  const uint32_t ring_s = smem_addr(smem) + warp * T::kStages * T::kTileBytes;
  const uint32_t header_s = smem_addr(mine), bar_s = header_s + 32 * T::kStages, query_s = header_s + T::kHeaders;
  Header* headers = reinterpret_cast<Header*>(mine);
  if constexpr (TMA) {
    if (lane == 0) {
      for (int i = 0; i < T::kStages; ++i) ptx::mbar_init(bar_s + 8 * i, 1);
      ptx::fence_mbar_init();
      ptx::fence_proxy_async_smem();
    }
    __syncwarp();
  }

  // ---- the load side: where the next tile lies
  int lb = b, llen = max(0, min(__ldg(a.seq_lens + b), a.max_len));
  int lt = static_cast<int>(tile0) * KT;     // first token of the next tile
  int lleft = static_cast<int>(left);
  bool seg_first = true, from_start = lt == 0;
  int q_slot = 0;
  // page and offset in it of token lt + lane (rows, cp.async) or lt + lane * box tokens (boxes, TMA)
  int pg, off;
  bool bad = false;
  const int step_log2 = TMA ? a.box_tokens_log2 : 0, steps = KT >> step_log2;
  auto look_up = [&]() {
    const int t = lt + (lane << step_log2);
    pg = -1;
    off = 0;
    if (lane < steps && t < llen) {
      const int p = static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(t)) * a.page_magic) >> a.page_shift);
      off = t - p * a.cache.page_size;
      pg = __ldg(a.table + lb * a.table_stride + p);
    }
  };
  look_up();

  auto issue = [&](int stage) {
    if (lleft > 0) {
      const bool inside = lane < steps && lt + (lane << step_log2) < llen;
      const bool ok = inside && pg >= 0 && pg < a.cache.num_pages;
      bad |= inside && !ok;
      unsigned mask = __ballot_sync(0xffffffffu, ok);
      const uint32_t ks = ring_s + stage * T::kTileBytes, vs = ks + KT * T::kRowK, qs = query_s + q_slot * a.q_bytes;
      const uint32_t bar = bar_s + 8 * stage;
      const bool ends = lt + KT >= llen;
      const uint8_t* qrow = a.q + lb * a.q_batch + static_cast<long long>(h0) * T::kRowK;
      if constexpr (TMA) {
        if (lane == 0) {
          const uint32_t bytes = (__popc(mask) << step_log2) * T::kKeyBytes + (seg_first ? nh * T::kRowK : 0);
          ptx::mbar_arrive_expect_tx(bar, bytes);
          if (seg_first) bulk_load(qs, qrow, nh * T::kRowK, bar);
        }
        __syncwarp();
        if (ok) {
          const int row = lane << step_log2;
          for (int c = 0; c < T::kRowK / kChunkBytes<T::kRowK>; c += a.box_chunks)
            tma_load_5d(ks + (c * KT + row) * kChunkBytes<T::kRowK>, &kmap, bar, 0, off, c, hk, pg);
          for (int c = 0; c < T::kRowV / kChunkBytes<T::kRowV>; c += a.box_chunks)
            tma_load_5d(vs + (c * KT + row) * kChunkBytes<T::kRowV>, &vmap, bar, 0, off, c, hk, pg);
        }
        mask = __ballot_sync(0xffffffffu, lane < KT && lt + lane < llen && ((mask >> (lane >> step_log2)) & 1));
      } else {
        const long long krow = ok ? pg * a.cache.k_page + off * a.cache.k_tok : 0;
        const long long vrow = ok ? pg * a.cache.v_page + off * a.cache.v_tok : 0;
#pragma unroll
        for (int i = 0; i < KT * kChunksK / 32; ++i) {
          const int x = i * 32 + lane, r = x / kChunksK, c = x % kChunksK;
          const long long o = __shfl_sync(0xffffffffu, krow, r);
          copy16(ks + place<T::kRowK, KT>(r, c), kbase + o + c * 16, (mask >> r) & 1 ? 16 : 0);
        }
#pragma unroll
        for (int i = 0; i < KT * kChunksV / 32; ++i) {
          const int x = i * 32 + lane, r = x / kChunksV, c = x % kChunksV;
          const long long o = __shfl_sync(0xffffffffu, vrow, r);
          copy16(vs + place<T::kRowV, KT>(r, c), vbase + o + c * 16, (mask >> r) & 1 ? 16 : 0);
        }
        if (seg_first)
          for (int x = lane; x < nh * kChunksK; x += 32) copy16(qs + x * 16, qrow + x * 16, 16);
      }
      if (lane == 0) {
        Header* h = headers + stage;
        const uint32_t s = header_s + stage * 32;
        h->mask = mask;
        h->b = lb;
        const bool last = ends || lleft == 1;
        h->q_slot = q_slot;
        h->flags = (seg_first ? kFirst : 0) | (last ? kLast : 0) | (from_start && ends ? kDirect : 0) | (from_start ? kSlot1 : 0);
        if (FP8 && seg_first) {
          const int di = a.desc_per_head ? lb * a.cache.H_kv + hk : 0;
          if (a.q_desc) copy4(s + 16, a.q_desc + di); else h->dq = 1.0f;
          if (a.k_desc) copy4(s + 20, a.k_desc + di); else h->dk = 1.0f;
          if (a.v_desc) copy4(s + 24, a.v_desc + di); else h->dv = 1.0f;
        }
      }
      // the tile after it
      if (seg_first) q_slot = q_slot + 1 == T::kStages - 1 ? 0 : q_slot + 1;
      --lleft;
      seg_first = false;
      lt += KT;
      if (ends && lleft > 0) {
        do {
          ++lb;
          llen = max(0, min(__ldg(a.seq_lens + lb), a.max_len));
        } while (llen == 0 && lb + 1 < a.B);
        lt = 0;
        seg_first = true;
        from_start = true;
      }
      if (lleft > 0) look_up();
    }
    copy_commit();
  };

  // ---- the compute side
  const int t4 = lane & 3, g8 = lane >> 2;
  // this lane's rows and halves in the ldmatrix reads of a K tile and of a (transposed) V tile
  const uint32_t k_lane = lane_part<T::kRowK>(lane & 15, lane >> 4);
  const uint32_t v_lane = FP8 ? lane_part<T::kRowV>(lane & 15, lane >> 4)
                              : lane_part<T::kRowV>((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1);
  uint32_t qf[NT][kKSteps][2];
  float o[NT][kMTiles][4], m[NT][2], l[NT][2];
  float scale = 0.0f, dv = 1.0f;
  constexpr float kLift = FP8 ? 15.0f : 0.0f;  // e4m3: weights in fp16 up to 2^15, so that light ones keep their bits

#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) issue(i);
  int stage = 0;
  uint32_t parity = 0;
  bool gave_up = false;
  // true once the stage's copies have landed; false after kWaitClocks without them
  auto arrived = [&](int st, uint32_t par) {
    const uint32_t bar = bar_s + 8 * st;
    bool done = ptx::mbar_try_wait(bar, par);
    if (!done) {
      const long long t0 = clock64();
      do done = ptx::mbar_try_wait(bar, par);
      while (!done && clock64() - t0 < kWaitClocks);
    }
    return static_cast<bool>(__all_sync(0xffffffffu, done));
  };
  for (int it = static_cast<int>(left); it > 0; --it) {
    if constexpr (TMA) {
      if (!arrived(stage, parity)) {
        gave_up = true;
        break;
      }
    } else {
      copy_wait<T::kStages - 2>();
    }
    __syncwarp();
    if constexpr (TMA && FP8) {
      if (headers[stage].flags & kFirst) {  // the descales came by cp.async
        copy_wait<0>();
        __syncwarp();
      }
    }
    const Header h = headers[stage];
    const uint32_t ks = ring_s + stage * T::kTileBytes, vs = ks + KT * T::kRowK;
    if (h.flags & kFirst) {
      const uint32_t qs = query_s + h.q_slot * a.q_bytes;
      scale = FP8 ? a.scale_log2 * h.dq * h.dk : a.scale_log2;
      dv = FP8 ? h.dv : 1.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < kMTiles; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
        // rows behind the last head repeat it: their columns are computed and never written
        const int r = min(n * 8 + (lane & 7), nh - 1);
#pragma unroll
        for (int i = 0; i < kKSteps; i += 2) {
          uint32_t x[4];
          ldsm4(qs + r * T::kRowK + (2 * i + (lane >> 3)) * 16, x);
          qf[n][i][0] = x[0];
          qf[n][i][1] = x[1];
          qf[n][i + 1][0] = x[2];
          qf[n][i + 1][1] = x[3];
        }
      }
    }
    // Refill the stage that the last iteration read.  At most kStages - 1 tiles are now ahead of the compute side, so as
    // many query slots are enough even if each begins another request: this one's queries are in registers.
    __syncwarp();
    issue(stage == 0 ? T::kStages - 1 : stage - 1);
    if (h.mask) {
      // S^T: rows are keys, columns heads; then scores in units of log2
      F2 x[KB][NT][2];
      const uint32_t kb_s = ks + k_lane;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float c[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kKSteps; ++i) {
          uint32_t r[4];
          ldsm4(lane_place<T::kRowK, KT>(kb_s, 2 * i, kb), r);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<kScoreKind>(c[n], r[0], r[1], r[2], r[3], qf[n][i][0], qf[n][i][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          x[kb][n][0] = mul2({c[n][0], c[n][1]}, {scale, scale});
          x[kb][n][1] = mul2({c[n][2], c[n][3]}, {scale, scale});
        }
      }
      if (h.mask != (KT == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (!((h.mask >> (kb * 16 + j * 8 + g8)) & 1))
#pragma unroll
              for (int n = 0; n < NT; ++n) x[kb][n][j] = {-INFINITY, -INFINITY};
        if constexpr (TMA) {  // whatever V holds behind the request's end is not a number to multiply by 0
          for (int i = lane; i < KT * kChunksV; i += 32)
            if (!((h.mask >> (i / kChunksV)) & 1)) ptx::st_shared_v4(vs + place<T::kRowV, KT>(i / kChunksV, i % kChunksV), 0, 0, 0, 0);
          ptx::fence_proxy_async_smem();  // before a later TMA load into this stage
          __syncwarp();
        }
      }
      // The reference m moves only when a key exceeds it: log2 of a weight is then above the lift.  (Before a segment's first
      // key m is -inf and every valid key's log2 weight +inf; each head has a valid key in this tile.)
      F2 y[KB][NT][2];
      float over = -INFINITY;
      auto weigh = [&]() {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              y[kb][n][j] = add2(x[kb][n][j], {kLift - m[n][0], kLift - m[n][1]});
              over = fmaxf(over, fmaxf(y[kb][n][j].x, y[kb][n][j].y));
            }
      };
      weigh();
      if (__any_sync(0xffffffffu, over > kLift)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = m[n][e];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
              t = e ? fmaxf(t, fmaxf(x[kb][n][0].y, x[kb][n][1].y)) : fmaxf(t, fmaxf(x[kb][n][0].x, x[kb][n][1].x));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float f = exp2_approx(m[n][e] - t);
            m[n][e] = t;
            l[n][e] *= f;
#pragma unroll
            for (int i = 0; i < kMTiles; ++i) {
              o[n][i][e] *= f;
              o[n][i][e + 2] *= f;
            }
          }
        weigh();
      }
      // weights, transposed into the B operand (keys are now the contraction)
      uint32_t pf[KB][NT][2];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const F2 w = {exp2_approx(y[kb][n][j].x), exp2_approx(y[kb][n][j].y)};
            const F2 sum = add2({l[n][0], l[n][1]}, w);
            l[n][0] = sum.x;
            l[n][1] = sum.y;
            pf[kb][n][j] = transpose8x8(pack2<FP8>(w.x, w.y));
          }
      // O^T += V^T P^T: rows are channels of V
      const uint32_t vb_s = vs + v_lane;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < kMTiles; i += 2) {
            // a register holds channels 2r, 2r+1 of two keys: the even channel is row r, the odd one row r + 8
            uint32_t r[4], v[8];
            ldsm4t(lane_place<T::kRowV, KT>(vb_s, i, kb), r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t q = __byte_perm(r[j], 0, 0x3120);
              v[2 * j] = widen(q);
              v[2 * j + 1] = widen_hi(q);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma<kValueKind>(o[n][i], v[0], v[1], v[2], v[3], pf[kb][n][0], pf[kb][n][1]);
              mma<kValueKind>(o[n][i + 1], v[4], v[5], v[6], v[7], pf[kb][n][0], pf[kb][n][1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kMTiles; ++i) {
            uint32_t r[4];
            ldsm4t(lane_place<T::kRowV, KT>(vb_s, 2 * i, kb), r);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma<kValueKind>(o[n][i], r[0], r[1], r[2], r[3], pf[kb][n][0], pf[kb][n][1]);
          }
        }
      }
    }
    if (h.flags & kLast) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[n][e];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          const int head = n * 8 + t4 * 2 + e;
          if (head < nh) {
            if (h.flags & kDirect) {
              const long long row = static_cast<long long>(h.b) * a.H + h0 + head;
              const float f = sum > 0.0f ? dv / sum : 0.0f;
              __nv_bfloat16* out = a.out + row * DV;
#pragma unroll
              for (int i = 0; i < kMTiles; ++i) {
                const float y0 = o[n][i][e] * f, y1 = o[n][i][e + 2] * f;
                if constexpr (FP8) {
                  *reinterpret_cast<__nv_bfloat162*>(out + i * 16 + 2 * g8) = __floats2bfloat162_rn(y0, y1);
                } else {
                  out[i * 16 + g8] = __float2bfloat16_rn(y0);
                  out[i * 16 + g8 + 8] = __float2bfloat16_rn(y1);
                }
              }
              if (a.lse && g8 == 0)
                a.lse[row] = sum > 0.0f ? (m[n][e] + log2f(sum) - kLift) * 0.69314718055994531f : -INFINITY;
            } else {
              const long long row = (static_cast<long long>(g) * 2 + (h.flags & kSlot1 ? 1 : 0)) * a.H + h0 + head;
              float* part = a.part + row * DV;
#pragma unroll
              for (int i = 0; i < kMTiles; ++i) {
                if constexpr (FP8) {
                  *reinterpret_cast<float2*>(part + i * 16 + 2 * g8) = make_float2(o[n][i][e] * dv, o[n][i][e + 2] * dv);
                } else {
                  part[i * 16 + g8] = o[n][i][e];
                  part[i * 16 + g8 + 8] = o[n][i][e + 2];
                }
              }
              if (g8 == 0) a.ml[row] = make_float2(m[n][e] - kLift, sum);
            }
          }
        }
    }
    if (++stage == T::kStages) {
      stage = 0;
      parity ^= 1;
    }
  }
  copy_wait<0>();
  if (gave_up) {  // copies still in flight write to this block's shared memory: wait for them, again for a bounded time
    for (int i = 0; i < T::kStages; ++i) {
      arrived(stage, parity);
      if (++stage == T::kStages) {
        stage = 0;
        parity ^= 1;
      }
    }
    if (lane == 0) atomicOr(a.status, zyfa::kStatusTimeoutBit);
  }
  if (bad) atomicOr(a.status, zyfa::kStatusBadPageBit);
}

// Joins the parts of the requests that several groups worked on, and writes the rows of empty requests: one block of W
// warps per (request, head).  The parts' maxima and sums are read first, all at once; then the warps add up every W-th part
// each, whose loads do not depend on one another, and meet in shared memory in a fixed order.
template <int DV, int W>
__global__ void __launch_bounds__(W * 32) join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int kThreads = W * 32, kVec = DV / 32;
  using Vec = typename std::conditional<kVec == 4, float4, float2>::type;
  __shared__ float s_o[W][DV], s_m[W], s_l[W];
  wait_for_predecessor();
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned p0 = a.starts[b], p1 = a.starts[b + 1], per = a.starts[a.B + 1];
  const long long row = static_cast<long long>(b) * a.H + h;
  if (p0 == p1) {
    for (int i = threadIdx.x; i < DV; i += kThreads) a.out[row * DV + i] = __float2bfloat16_rn(0.0f);
    if (a.lse && threadIdx.x == 0) a.lse[row] = -INFINITY;
    return;
  }
  const int g0 = static_cast<int>(p0 / per), n = static_cast<int>((p1 - 1) / per) - g0 + 1;
  if (n == 1) return;
  // part i: group g0 + i, its slot 1 (a request that begins there) for the first, else slot 0
  auto part = [&](int i) { return (static_cast<long long>(g0 + i) * 2 + (i == 0 ? 1 : 0)) * a.H + h; };
  float m = -INFINITY;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    m = fmaxf(m, a.ml[part(i)].x);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  if (lane == 0) s_m[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) m = fmaxf(m, s_m[i]);
  float l = 0.0f;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float2 x = a.ml[part(i)];
    l += x.x == -INFINITY ? 0.0f : x.y * exp2_approx(x.x - m);
  }
#pragma unroll
  for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) l += s_l[i];
  float o[kVec] = {};
#pragma unroll 8
  for (int i = warp; i < n; i += W) {
    const Vec x = *reinterpret_cast<const Vec*>(a.part + part(i) * DV + lane * kVec);
    const float top = a.ml[part(i)].x, e = top == -INFINITY ? 0.0f : exp2_approx(top - m);
    const float* y = reinterpret_cast<const float*>(&x);
#pragma unroll
    for (int j = 0; j < kVec; ++j) o[j] = fmaf(y[j], e, o[j]);
  }
#pragma unroll
  for (int j = 0; j < kVec; ++j) s_o[warp][lane * kVec + j] = o[j];
  __syncthreads();
  for (int i = threadIdx.x; i < DV; i += kThreads) {
    float x = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) x += s_o[j][i];
    a.out[row * DV + i] = __float2bfloat16_rn(l > 0.0f ? x / l : 0.0f);
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// ------------------------------------------------------------------------------------------------
// host side

long long round_up(long long x, long long n) { return (x + n - 1) / n * n; }

// Chunks of up to 16 query heads that the heads of one KV head are cut into, as equal as they come.
int chunks_of(int group) { return (group + 15) / 16; }

// Groups of `units` warps that work on a call: as many as are resident at once, and no more than there can be tiles.
long long groups_of(long long warps, long long units, long long tiles) { return std::max(1ll, std::min(warps / units, tiles)); }

long long tiles_at_most(int B, long long max_len, int keys) { return B * ((max_len + keys - 1) / keys); }

constexpr int kMaxDevices = 64;

// Boxes of `tokens` rows by `chunks` column chunks of one head and page.  The chunk dimension follows the tokens, so that
// a box lands as [chunk][token][CB].
bool make_map(CUtensorMap* m, const uint8_t* base, bool fp8, int row_bytes, const zyfa::CacheView& c, long long page, long long tok,
              long long head, int tokens, int chunks) {
  const int es = fp8 ? 1 : 2, cb = row_bytes % 128 == 0 ? 128 : 64;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(cb / es), static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(row_bytes / cb),
                              static_cast<cuuint64_t>(c.H_kv), static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(tok), static_cast<cuuint64_t>(cb), static_cast<cuuint64_t>(head),
                                 static_cast<cuuint64_t>(page)};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(cb / es), static_cast<cuuint32_t>(tokens), static_cast<cuuint32_t>(chunks), 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return zyfa::encode_tensor_map(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint8_t*>(base), dims,
                                 strides, box, estr, cb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, int smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <bool FP8, int DQK, int DV, int NT, bool TMA>
zyfa_status_t launch(DecodeArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  using T = Tile<FP8, DQK, DV>;
  a.q_bytes = static_cast<int>(round_up(a.chunk_heads * T::kRowK, 16));
  const int smem = kWarps * (T::kStages * T::kTileBytes + (T::kStages - 1) * a.q_bytes + T::kHeaders);
  // one wave of resident blocks: 228 KiB of shared memory per SM, 1 KiB of it taken per block
  const int fit = std::min(T::blocks(NT), 233472 / (smem + 1024));
  a.groups = static_cast<int>(groups_of(nsm * fit * kWarps, a.units, tiles_at_most(a.B, a.max_len, T::kKeys)));
  // workspace: plan, (m, l), O
  a.starts = reinterpret_cast<unsigned*>(ws);
  ws += round_up((a.B + 2ll) * 4, 256);
  a.ml = reinterpret_cast<float2*>(ws);
  ws += round_up(2ll * a.groups * a.H * 8, 256);
  a.part = reinterpret_cast<float*>(ws);
  // Few rows have many parts each: more warps per row.
  const unsigned rows = static_cast<unsigned>(a.B) * a.H;
  const bool few = rows <= 4u * nsm;
  static std::atomic<int> set[kMaxDevices];
  if (set[dev].load(std::memory_order_acquire) < smem) {
    // Both kernels ask for the largest share of shared memory: an SM changes the share only when it is empty, so blocks
    // launched beside a predecessor of another share would find too little (1.5 times the time, 128 requests).
    auto prefer = [](const void* f) {
      return cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) == cudaSuccess;
    };
    const void* main = reinterpret_cast<const void*>(&decode_kernel<FP8, DQK, DV, NT, TMA>);
    if (cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess || !prefer(main) ||
        !prefer(reinterpret_cast<const void*>(&join_kernel<DV, 4>)) || !prefer(reinterpret_cast<const void*>(&join_kernel<DV, 16>)))
      return ZYFA_ERR_CUDA;
    set[dev].store(smem, std::memory_order_release);
  }
  const long long warps = static_cast<long long>(a.groups) * a.units;
  cudaError_t e = launch_dependent(decode_kernel<FP8, DQK, DV, NT, TMA>, static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, smem,
                                   stream, a, kmap, vmap);
  if (e != cudaSuccess) return ZYFA_ERR_CUDA;
  e = few ? launch_dependent(join_kernel<DV, 16>, rows, 512, 0, stream, a) : launch_dependent(join_kernel<DV, 4>, rows, 128, 0, stream, a);
  return e == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
}

template <bool FP8, int DQK, int DV>
zyfa_status_t pick(DecodeArgs& a, const zyfa::CacheView& c, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  using T = Tile<FP8, DQK, DV>;
  CUtensorMap kmap, vmap;
  std::memset(&kmap, 0, sizeof(kmap));
  std::memset(&vmap, 0, sizeof(vmap));
  // Boxes: as many tokens of a page as divide both the page and the tile.  A broadcast (stride 0) or very large stride has no
  // tensor map, and a page of an odd size no boxes that fill the swizzle pattern (8 rows): those go row by row.
  int tokens = T::kKeys;
  while (tokens > 1 && c.page_size % tokens != 0) tokens /= 2;
  bool tma = tokens >= 8;
  for (long long s : {c.k_page, c.k_tok, c.k_head, c.v_page, c.v_tok, c.v_head}) tma = tma && s > 0 && s < (1ll << 40);
  a.box_tokens_log2 = tokens == 32 ? 5 : tokens == 16 ? 4 : 3;
  a.box_chunks = tokens == T::kKeys ? 3 : 1;  // at most three chunks in a row: one box, or one per chunk
  if (tma) {
    const int ck = T::kRowK / kChunkBytes<T::kRowK>, cv = T::kRowV / kChunkBytes<T::kRowV>;
    tma = make_map(&kmap, c.k, FP8, T::kRowK, c, c.k_page, c.k_tok, c.k_head, tokens, std::min(ck, a.box_chunks)) &&
          make_map(&vmap, c.v, FP8, T::kRowV, c, c.v_page, c.v_tok, c.v_head, tokens, std::min(cv, a.box_chunks));
  }
  const bool wide = a.chunk_heads > 8;
  if (tma)
    return wide ? launch<FP8, DQK, DV, 2, true>(a, kmap, vmap, nsm, dev, ws, stream)
                : launch<FP8, DQK, DV, 1, true>(a, kmap, vmap, nsm, dev, ws, stream);
  return wide ? launch<FP8, DQK, DV, 2, false>(a, kmap, vmap, nsm, dev, ws, stream)
              : launch<FP8, DQK, DV, 1, false>(a, kmap, vmap, nsm, dev, ws, stream);
}

}  // namespace

extern "C" {

size_t zyfa_attn_decode_paged_workspace_bytes(int B, int H, int H_kv, int D_v, long long max_len) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || (D_v != 64 && D_v != 128) || max_len < 0) return 0;
  const long long units = static_cast<long long>(H_kv) * chunks_of(H / H_kv);
  const long long groups = groups_of(kMaxSms * kMaxWarpsPerSm, units, tiles_at_most(B, max_len, 16));
  return static_cast<size_t>(round_up((B + 2ll) * 4, 256) + round_up(2 * groups * H * 8, 256) + 2 * groups * H * D_v * 4);
}

zyfa_status_t zyfa_attn_decode_paged(const void* q, long long q_batch_stride, const zyfa_paged_cache_t* cache,
                                     const int* block_table, long long table_stride, int max_pages,
                                     const int* seq_lens, void* out, float* lse, int B, int H, float softmax_scale,
                                     const float* q_descale, const float* k_descale, const float* v_descale,
                                     int descale_per_kv_head, void* workspace, size_t workspace_bytes,
                                     cudaStream_t stream) {
  using zyfa::aligned;
  DecodeArgs a = {};
  const zyfa_status_t st = zyfa::check_cache(cache, &a.cache);
  if (st != ZYFA_OK) return st;
  const int H_kv = cache->H_kv, D_qk = cache->D_qk, D_v = cache->D_v;
  const bool fp8 = cache->dtype == ZYFA_DTYPE_E4M3;
  const int es = zyfa::element_size(cache->dtype);
  if (B < 0 || H < 1 || H % H_kv != 0 || max_pages < 0 || table_stride < max_pages) return ZYFA_ERR_INVALID_ARG;
  if (descale_per_kv_head != 0 && descale_per_kv_head != 1) return ZYFA_ERR_INVALID_ARG;
  if (!std::isfinite(softmax_scale) || softmax_scale < 0.0f) return ZYFA_ERR_INVALID_ARG;
  if (q_batch_stride < 0) return ZYFA_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * cache->page_size > (1ll << 30)) return ZYFA_ERR_UNSUPPORTED;
  if (B > 65536 || H > 65536 || static_cast<long long>(B) * H > (1ll << 24)) return ZYFA_ERR_UNSUPPORTED;
  if (q_batch_stride > (1ll << 40)) return ZYFA_ERR_UNSUPPORTED;
  if (B * ((static_cast<long long>(max_pages) * cache->page_size + 15) / 16) > 0x7fffffffll) return ZYFA_ERR_UNSUPPORTED;
  if (B == 0) return ZYFA_OK;
  if (!q || !out || !seq_lens || (max_pages > 0 && !block_table)) return ZYFA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || (q_batch_stride * es) % 16 != 0 || !aligned(out, 16) || !aligned(seq_lens, 4) ||
      !aligned(block_table, 4) || !aligned(lse, 4) || !aligned(q_descale, 4) || !aligned(k_descale, 4) ||
      !aligned(v_descale, 4))
    return ZYFA_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < zyfa_attn_decode_paged_workspace_bytes(
                                          B, H, H_kv, D_v, static_cast<long long>(max_pages) * cache->page_size))
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
  a.desc_per_head = descale_per_kv_head;
  a.max_len = max_pages * cache->page_size;
  a.B = B;
  a.H = H;
  a.group = H / H_kv;
  a.chunks = chunks_of(a.group);
  a.chunk_heads = (a.group + a.chunks - 1) / a.chunks;
  a.units = H_kv * a.chunks;
  // t / page_size for t < 2^30: with s = ceil(log2 page_size) and M = floor(2^(30+s) / page_size) + 1 the error of
  // t M / 2^(30+s) is below 1 / page_size
  int s = 0;
  while ((1 << s) < cache->page_size) ++s;
  a.page_shift = 30 + s;
  a.page_magic = static_cast<uint32_t>((1ull << (30 + s)) / static_cast<unsigned>(cache->page_size) + 1);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (fp8)
    return D_qk == 64    ? pick<true, 64, 64>(a, a.cache, nsm, dev, ws, stream)
           : D_qk == 128 ? pick<true, 128, 128>(a, a.cache, nsm, dev, ws, stream)
                         : pick<true, 192, 128>(a, a.cache, nsm, dev, ws, stream);
  return D_qk == 64    ? pick<false, 64, 64>(a, a.cache, nsm, dev, ws, stream)
         : D_qk == 128 ? pick<false, 128, 128>(a, a.cache, nsm, dev, ws, stream)
                       : pick<false, 192, 128>(a, a.cache, nsm, dev, ws, stream);
}

}  // extern "C"
