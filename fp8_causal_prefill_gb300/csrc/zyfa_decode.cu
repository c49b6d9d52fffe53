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
// * The unit of work is a warp.  It streams its own tiles of KT keys through a private ring of cp.async stages and
//   shares nothing with other warps, so nothing in the loop waits for another warp.
// * Products run with the keys (or the channels of V) as the 16 rows of mma.m16n8k16 and the query heads as its 8
//   columns: S^T = K q^T, O^T = V^T P^T.  Groups of up to 8 heads waste no second half, K and V fragments come
//   straight from ldmatrix, and the accumulators of a 128-channel head take 32 registers.  An e4m3 cache is widened
//   to fp16 in registers (exact); P is held in fp16 lifted by 2^15 for e4m3, in bf16 otherwise.
// * Work is split over (request, key tile) evenly whatever the lengths: the tiles of all requests are numbered one after
//   the other and each group of warps (one warp per KV head and chunk of 16 query heads) takes an equal run
//   of them.  A group finds its run from seq_lens on the device, so the host never needs the lengths.  Heads of one
//   group read the same tokens at the same time, whose rows are neighbours in memory.
// * A request that lies in one group's run is written directly; otherwise each group leaves (m, l, O) of its
//   part in the workspace and a second kernel joins the parts in group order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "paged.cuh"

namespace {

constexpr int kWarps = 2;             // warps of a block; they never synchronise with one another
constexpr int kMaxSms = 160;          // the workspace is sized for at most this many SMs ...
constexpr int kMaxWarpsPerSm = 16;    // ... of this many warps
constexpr int kJoinThreads = 256;

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
  int q_bytes, ring_bytes;  // of a query slot, and of all a warp has in shared memory
  int* starts;   // [B + 2]: first tile of each request, then the total, then the tiles per group
  float2* ml;    // [groups][2][H]
  float* part;   // [groups][2][H][DV]
};

// ------------------------------------------------------------------------------------------------
// warp-level pieces

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

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
template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (FP8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
template <bool FP8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  if constexpr (FP8)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Where 16-byte chunk c of row r sits in a tile of ROW-byte rows: any 8 consecutive rows of one chunk column fall on
// 8 different 16-byte bank groups (rows of 128-byte multiples all start on the same group, others alternate between two).
template <int ROW>
__device__ __forceinline__ uint32_t place(int r, int c) {
  const int s = ROW % 128 == 0 ? (r & 7) : ((r >> 1) & 3);
  return static_cast<uint32_t>(r * ROW + ((c ^ s) << 4));
}

template <bool FP8, int DQK, int DV>
struct Tile {
  static constexpr int kEs = FP8 ? 1 : 2;
  static constexpr int kRowK = DQK * kEs, kRowV = DV * kEs;
  static constexpr int kKeyBytes = kRowK + kRowV;
  // Keys per stage, stages per warp and most blocks per SM (registers): a stage is at least 4 KiB, and the warps of an
  // SM together keep 100 KiB or more in flight.
  static constexpr int kKeys = kKeyBytes <= 128 ? 32 : 16;
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = kKeys * kKeyBytes;
  static constexpr int kHeaders = 128;
  static constexpr int blocks(int nt) { return nt == 1 ? (kKeyBytes <= 320 ? 8 : 4) : (kKeyBytes <= 320 ? 6 : 4); }
  static_assert(kStages * 32 <= kHeaders);
};

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
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int b) {
  const int len = max(0, min(__ldg(a.seq_lens + b), a.max_len));
  return (len + KT - 1) / KT;
}

template <bool FP8, int DQK, int DV, int NT>
__global__ void __launch_bounds__(kWarps * 32, (Tile<FP8, DQK, DV>::blocks(NT)))
    decode_kernel(const __grid_constant__ DecodeArgs a) {
  using T = Tile<FP8, DQK, DV>;
  constexpr int KT = T::kKeys, KB = KT / 16, es = T::kEs;
  constexpr int kChunksK = T::kRowK / 16, kChunksV = T::kRowV / 16;
  constexpr int kKSteps = DQK / 16, kMTiles = DV / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + warp;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this group's run of tiles
  long long total = 0;
  for (int b = lane; b < a.B; b += 32) total += tiles_of<KT>(a, b);
#pragma unroll
  for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(0xffffffffu, total, s);
  const int g = static_cast<int>(w / a.units), unit = static_cast<int>(w % a.units);
  const long long per = (total + a.groups - 1) / a.groups;
  long long first = g * per;
  long long left = g < a.groups ? min(per, total - first) : 0;
  const bool writes_plan = w == 0;
  if (left <= 0 && !writes_plan) return;

  int b = 0;
  long long tile0 = 0;  // tile of request b that the run begins with
  {
    long long before = 0;
    int found = -1;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      const int n = b0 + lane < a.B ? tiles_of<KT>(a, b0 + lane) : 0;
      long long incl = n;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += o;
      }
      if (writes_plan && b0 + lane < a.B) a.starts[b0 + lane] = static_cast<int>(before + incl - n);
      const unsigned hit = __ballot_sync(0xffffffffu, first < before + incl);
      if (hit && found < 0) {
        const int l = __ffs(hit) - 1;
        found = b0 + l;
        tile0 = first - __shfl_sync(0xffffffffu, before + incl - n, l);
        if (!writes_plan) break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    b = max(found, 0);
    if (writes_plan && lane == 0) {
      a.starts[a.B] = static_cast<int>(total);
      a.starts[a.B + 1] = static_cast<int>(per);
    }
    if (left <= 0) return;
  }

  const int hk = unit / a.chunks, chunk = unit % a.chunks;
  const int h0 = hk * a.group + chunk * a.chunk_heads;                     // first query head of this warp
  const int nh = min(a.chunk_heads, a.group - chunk * a.chunk_heads);      // and how many
  const uint8_t* kbase = a.cache.k + hk * a.cache.k_head;
  const uint8_t* vbase = a.cache.v + hk * a.cache.v_head;
  // headers, query slots (one fewer than stages: see the loop), stages of K and V rows
  uint8_t* mine = smem + warp * a.ring_bytes;
  Header* headers = reinterpret_cast<Header*>(mine);
  const uint32_t header_s = smem_addr(mine), query_s = header_s + T::kHeaders;
  const uint32_t ring_s = query_s + (T::kStages - 1) * a.q_bytes;

  // ---- the load side: where the next tile lies
  int lb = b, llen = max(0, min(__ldg(a.seq_lens + b), a.max_len));
  int lt = static_cast<int>(tile0) * KT;     // first token of the next tile
  int lleft = static_cast<int>(left);
  bool seg_first = true, from_start = lt == 0;
  int q_slot = 0;
  int pg, off;                                // page and offset in it of token lt + lane
  bool bad = false;
  auto look_up = [&]() {
    const int t = lt + lane;
    pg = -1;
    off = 0;
    if (lane < KT && t < llen) {
      const int p = static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(t)) * a.page_magic) >> a.page_shift);
      off = t - p * a.cache.page_size;
      pg = __ldg(a.table + lb * a.table_stride + p);
    }
  };
  look_up();

  auto issue = [&](int stage) {
    if (lleft > 0) {
      const bool inside = lane < KT && lt + lane < llen;
      const bool ok = inside && pg >= 0 && pg < a.cache.num_pages;
      bad |= inside && !ok;
      const unsigned mask = __ballot_sync(0xffffffffu, ok);
      const long long krow = ok ? pg * a.cache.k_page + off * a.cache.k_tok : 0;
      const long long vrow = ok ? pg * a.cache.v_page + off * a.cache.v_tok : 0;
      const uint32_t ks = ring_s + stage * T::kTileBytes, vs = ks + KT * T::kRowK;
#pragma unroll
      for (int i = 0; i < KT * kChunksK / 32; ++i) {
        const int x = i * 32 + lane, r = x / kChunksK, c = x % kChunksK;
        const long long o = __shfl_sync(0xffffffffu, krow, r);
        copy16(ks + place<T::kRowK>(r, c), kbase + o + c * 16, (mask >> r) & 1 ? 16 : 0);
      }
#pragma unroll
      for (int i = 0; i < KT * kChunksV / 32; ++i) {
        const int x = i * 32 + lane, r = x / kChunksV, c = x % kChunksV;
        const long long o = __shfl_sync(0xffffffffu, vrow, r);
        copy16(vs + place<T::kRowV>(r, c), vbase + o + c * 16, (mask >> r) & 1 ? 16 : 0);
      }
      const bool ends = lt + KT >= llen;
      if (seg_first) {
        const uint32_t qs = query_s + q_slot * a.q_bytes;
        const uint8_t* qrow = a.q + lb * a.q_batch + static_cast<long long>(h0) * T::kRowK;
        for (int x = lane; x < nh * kChunksK; x += 32) {
          const int r = x / kChunksK, c = x % kChunksK;
          copy16(qs + place<T::kRowK>(r, c), qrow + r * T::kRowK + c * 16, 16);
        }
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
  uint32_t qf[NT][kKSteps][2];
  float o[NT][kMTiles][4], m[NT][2], l[NT][2];
  float scale = 0.0f, dv = 1.0f;
  constexpr float kLift = FP8 ? 15.0f : 0.0f;  // e4m3: weights in fp16 up to 2^15, so that light ones keep their bits

#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) issue(i);
  int stage = 0;
  for (int it = static_cast<int>(left); it > 0; --it) {
    copy_wait<T::kStages - 2>();
    __syncwarp();
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
        for (int i = 0; i < kChunksK; i += 4) {
          uint32_t x[4];
          ldsm4(qs + place<T::kRowK>(r, i + (lane >> 3)), x);
          if constexpr (FP8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              qf[n][i + j][0] = widen(x[j]);
              qf[n][i + j][1] = widen_hi(x[j]);
            }
          } else {
            qf[n][i / 2][0] = x[0];
            qf[n][i / 2][1] = x[1];
            qf[n][i / 2 + 1][0] = x[2];
            qf[n][i / 2 + 1][1] = x[3];
          }
        }
      }
    }
    // Refill the stage that the last iteration read.  At most kStages - 1 tiles are now ahead of the compute side, so as
    // many query slots are enough even if each begins another request: this one's queries are in registers.
    __syncwarp();
    issue(stage == 0 ? T::kStages - 1 : stage - 1);
    // S^T: rows are keys, columns heads
    float sc[KB][NT][4];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
      for (int n = 0; n < NT; ++n) sc[kb][n][0] = sc[kb][n][1] = sc[kb][n][2] = sc[kb][n][3] = 0.0f;
      const int r = kb * 16 + (lane & 15);
#pragma unroll
      for (int c = 0; c < kChunksK; c += 2) {
        uint32_t x[4];
        ldsm4(ks + place<T::kRowK>(r, c + (lane >> 4)), x);
        if constexpr (FP8) {
          // a register holds 4 channels of a key; two of them are contraction indices 2t, 2t+1, the others 2t+8, 2t+9
          const uint32_t a0 = widen(x[0]), a1 = widen(x[1]), a2 = widen_hi(x[0]), a3 = widen_hi(x[1]);
          const uint32_t e0 = widen(x[2]), e1 = widen(x[3]), e2 = widen_hi(x[2]), e3 = widen_hi(x[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma<FP8>(sc[kb][n], a0, a1, a2, a3, qf[n][c][0], qf[n][c][1]);
            mma<FP8>(sc[kb][n], e0, e1, e2, e3, qf[n][c + 1][0], qf[n][c + 1][1]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<FP8>(sc[kb][n], x[0], x[1], x[2], x[3], qf[n][c / 2][0], qf[n][c / 2][1]);
        }
      }
    }
    // scores in units of log2; the reference moves only when a key exceeds it
    const bool full = h.mask == (KT == 32 ? 0xffffffffu : 0xffffu);
    bool over = false;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[kb][n][e] * scale;
          if (!full && !((h.mask >> (kb * 16 + g8 + (e >> 1) * 8)) & 1)) x = -INFINITY;
          sc[kb][n][e] = x;
          over |= x > m[n][e & 1];
        }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[0][n][e], sc[0][n][e + 2]);
          if constexpr (KB == 2) x = fmaxf(x, fmaxf(sc[1][n][e], sc[1][n][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[n][e], x);
          const float f = mn == -INFINITY ? 1.0f : exp2_approx(m[n][e] - mn);
          m[n][e] = mn;
          l[n][e] *= f;
#pragma unroll
          for (int i = 0; i < kMTiles; ++i) {
            o[n][i][e] *= f;
            o[n][i][e + 2] *= f;
          }
        }
    }
    // weights, transposed into the B operand (keys are now the contraction)
    uint32_t pf[KB][NT][2];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = sc[kb][n][e];
          p[e] = exp2_approx(x - m[n][e & 1] + kLift);
          if (!full && x == -INFINITY) p[e] = 0.0f;
        }
        l[n][0] += p[0] + p[2];
        l[n][1] += p[1] + p[3];
        pf[kb][n][0] = transpose8x8(pack2<FP8>(p[0], p[1]));
        pf[kb][n][1] = transpose8x8(pack2<FP8>(p[2], p[3]));
      }
    // O^T += V^T P^T: rows are channels of V
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < kMTiles; i += 2) {
          // a register holds channels 2r, 2r+1 of two keys: the even channel is row r, the odd one row r + 8
          uint32_t x[4];
          ldsm4t(vs + place<T::kRowV>(kb * 16 + (lane & 15), i + (lane >> 4)), x);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = __byte_perm(x[j], 0, 0x3120);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma<FP8>(o[n][i], widen(x[0]), widen_hi(x[0]), widen(x[1]), widen_hi(x[1]), pf[kb][n][0], pf[kb][n][1]);
            mma<FP8>(o[n][i + 1], widen(x[2]), widen_hi(x[2]), widen(x[3]), widen_hi(x[3]), pf[kb][n][0], pf[kb][n][1]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kMTiles; ++i) {
          uint32_t x[4];
          ldsm4t(vs + place<T::kRowV>(kb * 16 + (lane >> 4) * 8 + (lane & 7), 2 * i + ((lane >> 3) & 1)), x);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<FP8>(o[n][i], x[0], x[1], x[2], x[3], pf[kb][n][0], pf[kb][n][1]);
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
    stage = stage + 1 == T::kStages ? 0 : stage + 1;
  }
  copy_wait<0>();
  if (bad) atomicOr(a.status, zyfa::kStatusBadPageBit);
}

// Joins the parts of the requests that several groups worked on, and writes the rows of empty requests: one block per
// (request, head), whose warps take every 8th part and meet in shared memory in a fixed order.
template <int DV>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int kW = kJoinThreads / 32, kPer = DV / 32;
  __shared__ float s_o[kW][DV], s_m[kW], s_l[kW];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p0 = a.starts[b], p1 = a.starts[b + 1], per = a.starts[a.B + 1];
  const long long row = static_cast<long long>(b) * a.H + h;
  if (p0 == p1) {
    if (threadIdx.x < DV) a.out[row * DV + threadIdx.x] = __float2bfloat16_rn(0.0f);
    if (a.lse && threadIdx.x == 0) a.lse[row] = -INFINITY;
    return;
  }
  const int g0 = p0 / per, g1 = (p1 - 1) / per;
  if (g0 == g1) return;
  float m = -INFINITY, l = 0.0f, o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.0f;
#pragma unroll 4
  for (int g = g0 + warp; g <= g1; g += kW) {
    const long long r = (static_cast<long long>(g) * 2 + (g == g0 ? 1 : 0)) * a.H + h;
    const float2 ml = a.ml[r];
    const float mn = fmaxf(m, ml.x);
    const float f = mn == -INFINITY ? 0.0f : exp2_approx(m - mn), e = mn == -INFINITY ? 0.0f : exp2_approx(ml.x - mn);
    m = mn;
    l = l * f + ml.y * e;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + a.part[r * DV + i * 32 + lane] * e;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) s_o[warp][i * 32 + lane] = o[i];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x >= DV) return;
  float M = -INFINITY;
#pragma unroll
  for (int i = 0; i < kW; ++i) M = fmaxf(M, s_m[i]);
  float L = 0.0f, O = 0.0f;
#pragma unroll
  for (int i = 0; i < kW; ++i) {
    const float e = s_m[i] == -INFINITY ? 0.0f : exp2_approx(s_m[i] - M);
    L += s_l[i] * e;
    O += s_o[i][threadIdx.x] * e;
  }
  a.out[row * DV + threadIdx.x] = __float2bfloat16_rn(L > 0.0f ? O / L : 0.0f);
  if (a.lse && threadIdx.x == 0) a.lse[row] = L > 0.0f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
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

template <bool FP8, int DQK, int DV, int NT>
zyfa_status_t launch(DecodeArgs& a, int nsm, int dev, uint8_t* ws, cudaStream_t stream) {
  using T = Tile<FP8, DQK, DV>;
  a.q_bytes = static_cast<int>(round_up(a.chunk_heads * T::kRowK, 128));
  a.ring_bytes = T::kHeaders + (T::kStages - 1) * a.q_bytes + T::kStages * T::kTileBytes;
  const int smem = a.ring_bytes * kWarps;
  // one wave of resident blocks: 228 KiB of shared memory per SM, 1 KiB of it taken per block
  const int fit = std::min(T::blocks(NT), 233472 / (smem + 1024));
  a.groups = static_cast<int>(groups_of(nsm * fit * kWarps, a.units, tiles_at_most(a.B, a.max_len, T::kKeys)));
  // workspace: plan, (m, l), O
  a.starts = reinterpret_cast<int*>(ws);
  ws += round_up((a.B + 2ll) * 4, 256);
  a.ml = reinterpret_cast<float2*>(ws);
  ws += round_up(2ll * a.groups * a.H * 8, 256);
  a.part = reinterpret_cast<float*>(ws);
  static std::atomic<int> set[kMaxDevices];
  if (set[dev].load(std::memory_order_acquire) < smem) {
    if (cudaFuncSetAttribute(decode_kernel<FP8, DQK, DV, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return ZYFA_ERR_CUDA;
    set[dev].store(smem, std::memory_order_release);
  }
  const long long warps = static_cast<long long>(a.groups) * a.units;
  decode_kernel<FP8, DQK, DV, NT><<<static_cast<unsigned>((warps + kWarps - 1) / kWarps), kWarps * 32, smem, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ZYFA_ERR_CUDA;
  // the join's blocks may start before the first kernel ends; they wait for it (griddepcontrol.wait)
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.H);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<DV>, a) == cudaSuccess ? ZYFA_OK : ZYFA_ERR_CUDA;
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
  const bool wide = a.chunk_heads > 8;
#define ZYFA_DECODE(F, K, V) (wide ? launch<F, K, V, 2>(a, nsm, dev, ws, stream) : launch<F, K, V, 1>(a, nsm, dev, ws, stream))
  if (fp8) return D_qk == 64 ? ZYFA_DECODE(true, 64, 64) : D_qk == 128 ? ZYFA_DECODE(true, 128, 128) : ZYFA_DECODE(true, 192, 128);
  return D_qk == 64 ? ZYFA_DECODE(false, 64, 64) : D_qk == 128 ? ZYFA_DECODE(false, 128, 128) : ZYFA_DECODE(false, 192, 128);
#undef ZYFA_DECODE
}

}  // extern "C"
