// Causal attention over packed prompts, grouped heads.
//
//   o_i = sum_{j <= i + Lk - Lq} e^(s_ij - m_i) v_j / sum_j e^(s_ij - m_i)
//
// One CTA per SM at a time, which takes over the work of CTAs that have not
// started (cluster launch control), the longest rows first: dealt out in turn
// instead, the CTA with most to do had 18 to 54 % more than the mean.  A work
// item is one key head and a block of
// consecutive queries of one sequence; the G query heads of the key head and
// the block's tokens are the rows of two 128-row tiles (row = token * G +
// head), so a short prompt fills a tile with its heads and every key tile is
// read once for both tiles.  Per 128 keys and tile:
//   S = Q K^T     tcgen05, operands in shared memory, S fp32 in TMEM
//   P = e^(S - m) one thread per row, P written as bf16 over S in TMEM
//   O += P V      tcgen05, P from TMEM, V as it lies in memory (N-major)
// Warps 0-3 and 4-7 are the rows of tile 0 and 1, warp 8 issues the TMA
// loads (K and V tiles through one ring), warp 9 the products.  While one
// tile's exponentials run, the other tile's products do.
//
// m is the row maximum when it was last moved: O is rescaled only where the
// maximum has grown by more than 2^8 (the weights stay far inside bf16's and
// the sum inside fp32's range, and the quotient is the same), so the rescale
// through TMEM is rare.
//
// With too few blocks to fill the SMs evenly (few queries behind a long prefix)
// an item's key tiles are divided among several CTAs, whose outputs, maxima and sums a
// second kernel joins, a warp a row: 64 queries of 32 heads on 8, D = 128,
// behind 131072 keys 1851 -> 139 us, one query 1696 -> 121 us (its keys' and
// values' bytes alone 81 us), one query behind 2048 keys 37 -> 21 us.
//
// Rows that do not see a key must not feel its value, but 0 * NaN is NaN in a
// matrix product: warps 10-11 look at the V tiles that not every row sees whole.
// Rows behind the sequence's end are zeroed there, and so are values that are
// not finite, whose keys are listed; the rows that see such a key add its
// infinity or NaN to their outputs at the end.  So the bits of every other
// output are what they would be without it (16384 tokens, all values NaN: 1.26 ms,
// one key in a thousand infinite: as without).
//
// Measured: 16384 tokens, 16 heads on 2, D = 128: 0.89 ms in a short run (1230
// TFLOP/s, 0.75 of the measured bf16 product), 1.02 ms in a long one; a chunk of
// 8192 queries of 64 heads on 131072 keys 28 ms (1200 TFLOP/s).  What bounds it:
// with N = 128 the products with K alone read shared memory as long as they
// compute, next to the loads' writes and V (2048 cycles of each for the two
// tiles and 128 keys; measured 3800).  Tried and not kept: two 64-key score
// buffers a tile (1.11 ms: products with N = 64 read more than they compute), the
// product with V begun at half of the weights (0.93 ms), waits that spin.
// D = 64: 4 chunks of up to 2048 queries on up to 4548 keys 137 us; the weights
// bound it, an eighth of which the FMA pipes take (160 -> 152 us in a short run).
#include <cudaTypedefs.h>

#include <cmath>

#include "../../include/ai_index.h"
#include "common.cuh"
#include "kernels.h"

namespace aiidx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct PromptArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;  // strides, elements
  const int32_t* cu_q;
  const int32_t* cu_k;
  int n_seqs, total_q, total_k, Hq, Hkv, G;
  float c2;  // scale * log2 e
  uint16_t* out;
  float* lse;
  int32_t* status;
};

int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

// A sequence's rows; false (and flagged) where the offsets are not ascending
// within the totals.
__device__ __forceinline__ bool seq_rows(const PromptArgs& a, int b, int* q0, int* lq, int* k0, int* lk) {
  *q0 = a.cu_q[b];
  *k0 = a.cu_k[b];
  const int q1 = a.cu_q[b + 1], k1 = a.cu_k[b + 1];
  *lq = q1 - *q0;
  *lk = k1 - *k0;
  const bool ok = *q0 >= 0 && q1 >= *q0 && q1 <= a.total_q && *k0 >= 0 && k1 >= *k0 && k1 <= a.total_k;
  if (!ok) atomicOr(a.status, AI_DEVFLAG_RANGE);
  return ok;
}

// ------------------------------------------------------------ tensor cores
constexpr int kTile = 128;        // rows of a query tile, keys of a key tile
constexpr int kThreads = 384;
template <int D>
constexpr int kPolyOf = D == 64 ? 1 : 0;      // pairs of weights in eight that the FMA pipes compute
constexpr float kGrow = 8.f;      // log2 by which the maximum may grow before O is rescaled

template <int D>
struct Smem {
  static constexpr int kHalves = D / 64;          // 64-element (128-byte) column blocks
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kSlots = D == 128 ? 5 : 8; // ring of K and V tiles
  static constexpr int kBars = 4 + 4 * kSlots + 6 + 4;
  // lists of values that are not finite: of so many items (next_read holds the
  // loads to two items ahead of the slowest warp) and, of each, so many tiles that
  // not every row sees whole (its queries see up to 255 keys more than its first)
  static constexpr int kLists = 4, kPartly = 3;
  static constexpr int kBytes = 1024 + (2 + kSlots) * kTileBytes + kBars * 8 + 16 + 32 + kLists * kPartly * 16 + 8;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// TMEM columns: the two score tiles (their weights over them), the two outputs.
constexpr uint32_t kColS = 0, kColO = 256;

// One work item.
struct Item {
  int head, qtok, n_tok;      // key head, first query row, queries in the block (0: nothing to do)
  int k0, lk;                 // first key row, keys of the sequence
  int see0;                   // keys that the block's first query sees (may be <= 0)
  int j0;                     // first key tile of this CTA's part
  int tiles[2];               // key tiles of the part that each query tile needs
  __device__ int see(int tok) const { return max(0, min(lk, see0 + tok)); }
  __device__ int n() const { return max(tiles[0], tiles[1]); }
  // the part's first key tile that some row does not see all of
  __device__ int first_mixed() const { return max(0, see(0) / kTile - j0); }
  __device__ bool mixed(int j) const { return (j0 + j + 1) * kTile > see(0); }
};

struct Schedule {
  int n_slots, qb, tpt;       // slots per key head, queries per block and per tile
  int64_t n_items;
  int n_split;                // parts of an item's key tiles
  float2* ml;                 // n_split > 1: [n_items][n_split][256] maximum, sum
  float* o;                   //              [n_items][n_split][256][D] output before the division
};
constexpr int kMaxSplit = 128;
constexpr int kMaxTokens = 0x7fffffff - 2 * kTile;

// Slot s belongs to the last sequence b with cu_q[b] / qb + b <= s: each
// sequence has at least as many slots as blocks.
__device__ Item whole_item(const PromptArgs& a, const Schedule& sc, int64_t it) {
  Item x;
  x.j0 = 0;
  x.head = static_cast<int>(it % a.Hkv);
  const int slot = sc.n_slots - 1 - static_cast<int>(it / a.Hkv);  // the longest rows first
  int lo = 0, hi = a.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_q[mid] / sc.qb + mid <= slot) lo = mid;
    else hi = mid;
  }
  x.n_tok = 0;
  x.tiles[0] = x.tiles[1] = 0;
  int q0, lq;
  if (!seq_rows(a, lo, &q0, &lq, &x.k0, &x.lk)) return x;
  const int blk = slot - (q0 / sc.qb + lo);
  const int64_t first = static_cast<int64_t>(blk) * sc.qb;
  if (blk < 0 || first >= lq) return x;
  x.qtok = q0 + static_cast<int>(first);
  x.n_tok = static_cast<int>(min(static_cast<int64_t>(sc.qb), lq - first));
  x.see0 = static_cast<int>(max(static_cast<int64_t>(x.lk) - lq + first + 1, static_cast<int64_t>(-(1 << 30))));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int last = min((i + 1) * sc.tpt, x.n_tok) - 1;
    x.tiles[i] = last >= i * sc.tpt ? (x.see(last) + kTile - 1) / kTile : 0;
  }
  return x;
}
// The work of block `it`: part it % n_split of item it / n_split.
template <bool kSplit>
__device__ Item item_at(const PromptArgs& a, const Schedule& sc, int64_t it) {
  if (!kSplit) return whole_item(a, sc, it);
  const int part = static_cast<int>(it % sc.n_split);
  Item x = whole_item(a, sc, it / sc.n_split);
  const int64_t n = x.n();
  x.j0 = static_cast<int>(n * part / sc.n_split);
  const int j1 = static_cast<int>(n * (part + 1) / sc.n_split);
#pragma unroll
  for (int i = 0; i < 2; ++i) x.tiles[i] = max(0, min(x.tiles[i], j1) - x.j0);
  return x;
}

// Asks for the work of a CTA that has not started; the answer (16 bytes)
// completes on the barrier.
__device__ __forceinline__ void take_request(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// The item taken over, or -1 where none was left.
__device__ __forceinline__ int64_t take_answer(const uint4* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 h;\n .reg .b32 y, z, w;\n ld.shared.b128 h, [%2];\n mov.u32 %1, 0;\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n}\n"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? static_cast<int64_t>(x) : -1;
}

// Matrix descriptor of an operand that lies N-major (rows of K, 64 elements
// of N per 128-byte row): 8-row groups 1024 bytes apart along K, 64-element
// column blocks `block` bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t block) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// D[tmem] (+)= A[tmem] * B[smem].
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Pairs of floats in a 64-bit register, for the two-wide fp32 instructions.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t exp2_mufu2(uint64_t x) { return f2(ex2(lo_of(x)), ex2(hi_of(x))); }
// 2^x for x <= 2^7 on the FMA pipes, which the sixteen exponentials a cycle of
// the special function units would leave idle: x = n + f with f in [-1/2, 1/2]
// (rounded by adding 1.5 2^23), 2^f by the polynomial of degree 5 that
// interpolates it at the Chebyshev nodes (2.1e-7 with its fp32 rounding), 2^n
// from the exponent bits.  Below -127 the result is 0; NaN stays NaN.
__device__ __forceinline__ float floor127(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fC2FE0000;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x) {
  constexpr float kRound = 12582912.f + 127.f;
  const uint64_t y = f2(floor127(lo_of(x)), floor127(hi_of(x)));
  const uint64_t t = add2(y, f2(kRound, kRound));
  const uint64_t f = add2(y, mul2(add2(t, f2(-kRound, -kRound)), f2(-1.f, -1.f)));
  uint64_t p = fma2(f, f2(0.00133908634f, 0.00133908634f), f2(0.00967603192f, 0.00967603192f));
  p = fma2(p, f, f2(0.0555035711f, 0.0555035711f));
  p = fma2(p, f, f2(0.240221075f, 0.240221075f));
  p = fma2(p, f, f2(0.693147188f, 0.693147188f));
  p = fma2(p, f, f2(1.00000008f, 1.00000008f));
  return mul2(p, f2(__uint_as_float(static_cast<uint32_t>(t) << 23), __uint_as_float(static_cast<uint32_t>(t >> 32) << 23)));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p != 0;
}

// Adds to columns [c, c + 32) of a row's output the values that are not finite
// of the listed keys that it sees: their weight is positive, so what matters is
// their sign.  Bit b of list[q][u]: key u + 8 b of the part's key tile j + q.
__device__ __forceinline__ void add_listed(const PromptArgs& a, const Item& x, const uint16_t (*list)[8], int j, int n,
                                           int see, int c, float* y) {
  for (int q = 0; j + q < n; ++q) {
    for (int u = 0; u < 8; ++u) {
      for (uint32_t bits = list[q][u]; bits; bits &= bits - 1) {
        const int key = (x.j0 + j + q) * kTile + u + 8 * (__ffs(bits) - 1);
        if (key >= see) continue;
        const uint4* v = reinterpret_cast<const uint4*>(a.v + (x.k0 + key) * a.v_tok + x.head * a.v_head + c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = v[i];
          const uint32_t pair[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int h = 0; h < 8; ++h) {
            const float f = __uint_as_float(h & 1 ? pair[h / 2] & 0xffff0000u : pair[h / 2] << 16);
            if (f - f != 0.f) y[i * 8 + h] += f;
          }
        }
      }
    }
  }
}

template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    k_prompt_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const PromptArgs a, const Schedule sc) {
  using L = Smem<D>;
  constexpr int kSlots = L::kSlots, kPoly = kPolyOf<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sq = base;                              // [2] query tiles
  uint8_t* ring = base + 2 * L::kTileBytes;        // [kSlots] key / value tiles
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kSlots * L::kTileBytes);
  uint64_t* q_full = bars;                         // [2] query tile landed
  uint64_t* q_empty = bars + 2;                    // [2] last product that reads it done
  uint64_t* kv_full = bars + 4;                    // [kSlots] key tile, or V tile that every row sees whole
  uint64_t* kv_empty = kv_full + kSlots;
  uint64_t* mx_full = kv_empty + kSlots;           // [kSlots] V tile that some row sees in part
  uint64_t* v_clean = mx_full + kSlots;            // [kSlots] and looked at
  uint64_t* s_full = v_clean + kSlots;             // [2] scores in TMEM
  uint64_t* p_full = s_full + 2;                   // [2] weights in TMEM
  uint64_t* o_full = p_full + 2;                   // [2] last product with V of an item done
  uint64_t* next_full = o_full + 2;                // [2] next item known
  uint64_t* next_read = next_full + 2;             // [2] and read by every warp
  uint4* answer = reinterpret_cast<uint4*>((reinterpret_cast<uintptr_t>(next_read + 2) + 15) & ~uintptr_t(15));  // [2]
  // [kLists][kPartly][8], see add_listed
  uint16_t (*lists)[L::kPartly][8] = reinterpret_cast<uint16_t (*)[L::kPartly][8]>(answer + 2);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(lists + L::kLists);
  int* abort = reinterpret_cast<int*>(tmem_slot + 1);
  int* err = a.status;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&next_full[i], 1);
      mbar_init(&next_read[i], kThreads / 32);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&mx_full[s], 1);
      mbar_init(&v_clean[s], 2);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  dependency_wait();
  const uint32_t tmem = *tmem_slot;
  // the item after this warp's r-th; -1: no more
  auto next_item = [&](uint32_t r) {
    const uint32_t b = r & 1;
    if (!__all_sync(0xffffffffu, mbar_wait(&next_full[b], (r >> 1) & 1, err, abort))) return static_cast<int64_t>(-1);
    const int64_t it = take_answer(&answer[b]);
    fence_proxy_async_smem();   // before the next answer lands there
    __syncwarp();
    if (lane == 0) mbar_arrive(&next_read[b]);
    return it;
  };

  // the rows' warps take registers that the others do not need (8 x 208 + 4 x
  // 88 a lane, as many as the block was launched with: 12 x 168)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      // ---------------------------------------------------------- TMA loads
      const bool leader = elect_one();
      uint32_t g = 0, nq[2] = {0, 0};
      // by slot: parity of the next phase of its two barriers, and which one
      // its last load completes on
      uint32_t kv_next = 0, mx_next = 0, last_mx = 0;
      bool ok = true;
      auto all = [&](bool x) { return __all_sync(0xffffffffu, x); };
      uint32_t r = 0;
      for (int64_t it = blockIdx.x; ok && it >= 0; ++r) {
        // the next item is asked for while this one is loaded
        if (r >= 2 && !all(mbar_wait(&next_read[r & 1], ((r >> 1) - 1) & 1, err, abort))) break;
        if (leader) take_request(&answer[r & 1], &next_full[r & 1]);
        const Item x = item_at<kSplit>(a, sc, it);
        for (int i = 0; ok && i < 2; ++i) {
          if (x.tiles[i] == 0) continue;
          if (nq[i] > 0 && !all(mbar_wait(&q_empty[i], (nq[i] - 1) & 1, err, abort))) {
            ok = false;
            break;
          }
          if (leader) {
            mbar_arrive_expect_tx(&q_full[i], sc.tpt * a.G * D * 2);
            for (int c = 0; c < L::kHalves; ++c)
              tma_load_3d(sq + i * L::kTileBytes + c * (kTile * 128), &map_q, c * 64, x.head * a.G, x.qtok + i * sc.tpt,
                          &q_full[i]);
          }
          ++nq[i];
        }
        const int n = x.n();
        for (int t = 0; ok && t < 2 * n; ++t, ++g) {  // K 0, V 0, K 1, V 1, ..
          const int s = g % kSlots;
          if (g >= kSlots && !all(mbar_wait(&kv_empty[s], (g / kSlots - 1) & 1, err, abort))) {
            ok = false;
            break;
          }
          const bool mx = (t & 1) && x.mixed(t >> 1);
          uint64_t* full = mx ? &mx_full[s] : &kv_full[s];
          if (mx) {
            mx_next ^= 1u << s;
            last_mx |= 1u << s;
          } else {
            kv_next ^= 1u << s;
            last_mx &= ~(1u << s);
          }
          if (leader) {
            mbar_arrive_expect_tx(full, L::kTileBytes);
            for (int c = 0; c < L::kHalves; ++c)
              tma_load_3d(ring + s * L::kTileBytes + c * (kTile * 128), t & 1 ? &map_v : &map_k, c * 64, x.head,
                          x.k0 + (x.j0 + (t >> 1)) * kTile, full);
          }
        }
        if (ok) it = next_item(r);
      }
      if (*reinterpret_cast<volatile int*>(abort)) {
        // copies that this warp asked for may still be landing: bounded waits
        for (uint32_t s = 0; s < min(g, static_cast<uint32_t>(kSlots)); ++s) {
          const bool mx = (last_mx >> s) & 1;
          mbar_drain(mx ? &mx_full[s] : &kv_full[s], (((mx ? mx_next : kv_next) >> s) & 1) ^ 1);
        }
        for (int i = 0; i < 2; ++i)
          if (nq[i] > 0) mbar_drain(&q_full[i], (nq[i] - 1) & 1);
        if (r > 0) mbar_drain(&next_full[(r - 1) & 1], ((r - 1) >> 1) & 1);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ----------------------------------------------------------- products
      // The whole warp follows the loop and one elected lane issues: the operands
      // stay in uniform registers (issued from a one-lane branch, each product
      // first moved its descriptors there: 4700 cycles a tile pair for what the
      // tensor cores do in 2048).
      constexpr uint32_t id_s = idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t id_o = idesc_bf16_f32(kTile, D) | (1u << 16);  // B is N-major
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = sdesc_sw128(smem_u32(sq)), k_desc = sdesc_sw128(smem_u32(ring));
      const uint64_t v_desc = sdesc_sw128_mn(smem_u32(ring), kTile * 128);
      constexpr uint32_t kTileStep = L::kTileBytes >> 4;   // in descriptor units
      uint32_t slot = 0, nq[2] = {0, 0}, np[2] = {0, 0}, clean = 0, full = 0;  // next slot and parities by slot
      bool ok = true;
      auto all = [&](bool x) { return __all_sync(0xffffffffu, x); };
      auto wait_slot = [&](uint32_t s) {
        const uint32_t parity = (full >> s) & 1;
        full ^= 1u << s;
        return all(mbar_wait(&kv_full[s], parity, err, abort));
      };
      auto after = [&](uint32_t s) { return s + 1 == kSlots ? 0 : s + 1; };
      auto scores = [&](int i, uint32_t s) {  // S_i = Q_i K^T
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            constexpr uint32_t kHalf = kTile * 128 >> 4;
            const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 2;
            umma_bf16(tm + kColS + i * 128, q_desc + (i * kTileStep + off), k_desc + (s * kTileStep + off), id_s, kk > 0);
          }
          umma_commit(&s_full[i]);
        }
      };
      auto outputs = [&](int i, uint32_t s, bool first, bool last) {  // O_i (+)= P_i V
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_bf16_ta(tm + kColO + i * 128, tm + kColS + i * 128 + kk * 8,
                         v_desc + (s * kTileStep + kk * (16 * 128 >> 4)), id_o, !first || kk > 0);
          if (last) umma_commit(&o_full[i]);
        }
      };
      auto commit = [&](uint64_t* bar) {
        if (leader) umma_commit(bar);
      };
      uint32_t r = 0;
      for (int64_t it = blockIdx.x; ok && it >= 0; it = next_item(r++)) {
        const Item x = item_at<kSplit>(a, sc, it);
        const int n = x.n();
        if (n == 0) continue;
        ok = wait_slot(slot);
        for (int i = 0; ok && i < 2; ++i) {
          if (x.tiles[i] == 0) continue;
          if (!all(mbar_wait(&q_full[i], nq[i] & 1, err, abort))) {
            ok = false;
            break;
          }
          ++nq[i];
          tc_fence_after();
          scores(i, slot);
          if (x.tiles[i] == 1) commit(&q_empty[i]);
        }
        if (!ok) break;
        commit(&kv_empty[slot]);
        slot = after(slot);
        for (int j = 0; ok && j < n; ++j) {
          const uint32_t sv = slot, sk = after(slot);
          if (x.mixed(j)) {
            ok = all(mbar_wait(&v_clean[sv], (clean >> sv) & 1, err, abort));
            clean ^= 1u << sv;
          } else {
            ok = wait_slot(sv);
          }
          if (ok && j + 1 < n) ok = wait_slot(sk);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok) break;
            if (j < x.tiles[i]) {
              if (!all(mbar_wait(&p_full[i], np[i] & 1, err, abort))) {
                ok = false;
                break;
              }
              ++np[i];
              tc_fence_after();
              outputs(i, sv, j == 0, j + 1 == x.tiles[i]);
            }
            if (i == 1) commit(&kv_empty[sv]);
            if (j + 1 < x.tiles[i]) {
              scores(i, sk);
              if (j + 2 == x.tiles[i]) commit(&q_empty[i]);
            }
            if (i == 1 && j + 1 < n) commit(&kv_empty[sk]);
          }
          slot = j + 1 < n ? after(sk) : sk;
        }
      }
      // every product issued has completed before the TMEM is released
      for (int i = 0; i < 2; ++i) {
        if (nq[i] > 0) mbar_drain(&o_full[i], (nq[i] - 1) & 1);
        if (*reinterpret_cast<volatile int*>(abort) && nq[i] > 0) mbar_drain(&s_full[i], np[i] & 1);
      }
      __syncwarp();
    } else {
      // ------------------------------------------- V tiles that are seen in part
      const int t = threadIdx.x - 320;
      uint32_t g = 0, full = 0;
      int item = 0;
      bool ok = true;
      if (blockIdx.x == 0)  // every sequence's offsets, whatever the schedule reaches
        for (int b = t; b < a.n_seqs; b += 64) {
          int q0, lq, k0, lk;
          seq_rows(a, b, &q0, &lq, &k0, &lk);
        }
      uint32_t r = 0;
      for (int64_t it = blockIdx.x; ok && it >= 0; it = next_item(r++)) {
        const Item x = item_at<kSplit>(a, sc, it);
        const int n = x.n(), first = x.first_mixed();
        for (int j = first; ok && j < n; ++j) {
          const uint32_t e = g + 2 * j + 1;
          const int s = e % kSlots;
          // (these warps have nothing to do until an item's last tiles: a long row's time)
          ok = __all_sync(0xffffffffu, mbar_wait(&mx_full[s], (full >> s) & 1, err, abort, kSpinLimit << 6));
          if (!ok) break;
          full ^= 1u << s;
          const int lo = max(0, x.see(0) - (x.j0 + j) * kTile), hi = min(kTile, x.lk - (x.j0 + j) * kTile);
          uint32_t bad = 0;    // bit b: row t / 8 + 8 b
          // 16-byte unit u of the tile: row (u / 8) % 128; the swizzle stays within a row
          for (int u = t; u < L::kTileBytes / 16; u += 64) {
            const int row = (u >> 3) & (kTile - 1);
            uint4* p = reinterpret_cast<uint4*>(ring + s * L::kTileBytes) + u;
            if (row >= hi) {
              *p = make_uint4(0, 0, 0, 0);
            } else if (row >= lo) {
              const uint4 w = *p;
              // the carry out of an exponent of ones: infinity or NaN
              auto odd = [](uint32_t y) { return ((y & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
              const uint4 o = make_uint4(odd(w.x), odd(w.y), odd(w.z), odd(w.w));
              if (o.x | o.y | o.z | o.w) {
                bad |= 1u << (row >> 3);
                auto rest = [](uint32_t y, uint32_t z) { return y & ~((z >> 15) * 0xffffu); };
                *p = make_uint4(rest(w.x, o.x), rest(w.y, o.y), rest(w.z, o.z), rest(w.w, o.w));
              }
            }
          }
          // a row's units are eight lanes'
          for (int i = 1; i < 8; i <<= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, i);
          if ((t & 7) == 0) lists[item % L::kLists][j - first][t >> 3] = static_cast<uint16_t>(bad);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_clean[s]);
        }
        g += 2 * n;
        item += n > 0;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax
    const int i = warp >> 2;                         // query tile
    const int row = (warp & 3) * 32 + lane;          // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + kColS + i * 128 + lane_off, to = tmem + kColO + i * 128 + lane_off;
    const int tok = i * sc.tpt + row / a.G, gh = row % a.G;
    const bool used = row < sc.tpt * a.G;
    uint32_t np = 0, no = 0;   // score tiles, items with any
    int item = 0;
    bool ok = true;
    uint32_t r = 0;
    for (int64_t it = blockIdx.x; ok && it >= 0; it = next_item(r++)) {
      const Item x = item_at<kSplit>(a, sc, it);
      const int n = x.tiles[i];
      const int see = x.see(tok);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++np) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[i], np & 1, err, abort));
        if (!ok) break;
        tc_fence_after();
        const int limit = see - (x.j0 + j) * kTile;
        const bool part = (x.j0 + j + 1) * kTile > x.see(i * sc.tpt);  // warp-uniform
        float v[kTile];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, v + c * 32);
        tmem_ld_wait();
        if (part) {
#pragma unroll
          for (int u = 0; u < kTile; ++u) v[u] = u < limit ? v[u] : -INFINITY;
        }
        float mx4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int u = 4; u < kTile; u += 8) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            mx4[w] = u + 4 + w < kTile ? fmaxf(fmaxf(v[u + w], v[u + 4 + w]), mx4[w]) : fmaxf(v[u + w], mx4[w]);
        }
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const float want = mx == -INFINITY ? -INFINITY : mx * a.c2;
        const bool move = j == 0 || want > m + kGrow;
        if (j == 0) {
          m = want;
        } else if (__any_sync(0xffffffffu, move)) {
          const float mz = move ? want : m;
          const float f = move ? ex2(m - mz) : 1.f;  // m = -inf: nothing seen so far, O and l are 0
          // (these scores were issued after the last product with V and have
          // arrived, so O is complete)
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            float y[16];
            uint32_t w[16];
            tmem_ld16(to + c * 16, y);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 16; ++u) w[u] = __float_as_uint(y[u] * f);
            tmem_st16(to + c * 16, w);
          }
          l *= f;
          m = mz;
        }
        const float mu = m == -INFINITY ? 0.f : m;
        // weights: of eight pairs kPoly by polynomial, the rest by ex2
        uint64_t sum[2] = {0, 0};
        const uint64_t c2 = f2(a.c2, a.c2), nmu = f2(-mu, -mu);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const uint64_t x = fma2(f2(v[c * 32 + 2 * u], v[c * 32 + 2 * u + 1]), c2, nmu);
            const uint64_t e = (u % 8) * kPoly / 8 != (u % 8 + 1) * kPoly / 8 ? exp2_poly2(x) : exp2_mufu2(x);
            sum[u & 1] = add2(sum[u & 1], e);
            w[u] = pack2(lo_of(e), hi_of(e));
          }
          tmem_st16(ts + c * 16, w);  // over scores that are read already
        }
        const uint64_t total = add2(sum[0], sum[1]);
        l += lo_of(total) + hi_of(total);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[i]);  // (128 arrivals on one barrier queue up)
      }
      if (!ok) break;
      if (n > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[i], no & 1, err, abort));
        ++no;
        if (!ok) break;
        tc_fence_after();
      }
      const bool mine = used && tok < x.n_tok;
      // the tiles that this one's products have read, whose lists are written
      const uint16_t (*list)[8] = lists[item % L::kLists];
      const int first = x.first_mixed();
      uint32_t listed = 0;
      for (int q = 0; first + q < n; ++q) {
        const uint4 w = *reinterpret_cast<const uint4*>(list[q]);
        listed |= w.x | w.y | w.z | w.w;
      }
      if (kSplit) {
        // this part's share of the rows, for the joining kernel
        const int64_t at = it * (2 * kTile) + i * kTile + row;
        if (mine) sc.ml[at] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          if (n == 0) break;
          tmem_ld32(to + c * 32, v);
          tmem_ld_wait();
          if (listed) add_listed(a, x, list, first, n, see, c * 32, v);
          if (mine && l != 0.f) {
#pragma unroll
            for (int u = 0; u < 32; u += 4)
              *reinterpret_cast<float4*>(sc.o + at * D + c * 32 + u) = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
          }
        }
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* out = a.out + (static_cast<int64_t>(x.qtok + tok) * a.Hq + x.head * a.G + gh) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float v[32];
          if (n > 0) {
            tmem_ld32(to + c * 32, v);
            tmem_ld_wait();
            if (listed) add_listed(a, x, list, first, n, see, c * 32, v);
          }
          if (mine) {
            // a row that sees nothing is zero even where its tile computed something
#pragma unroll
            for (int u = 0; u < 32; u += 8) {
              uint4 w = make_uint4(0, 0, 0, 0);
              if (l != 0.f)
                w = make_uint4(pack2(v[u] * inv, v[u + 1] * inv), pack2(v[u + 2] * inv, v[u + 3] * inv),
                               pack2(v[u + 4] * inv, v[u + 5] * inv), pack2(v[u + 6] * inv, v[u + 7] * inv));
              *reinterpret_cast<uint4*>(out + c * 32 + u) = w;
            }
          }
        }
        if (mine && a.lse)
          a.lse[static_cast<int64_t>(x.qtok + tok) * a.Hq + x.head * a.G + gh] =
              l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      item += x.n() > 0;
      tc_fence_before();  // O is read before the next item's first product writes it
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of items (n_split > 1): a warp per row.
template <int D>
__global__ void __launch_bounds__(256) k_prompt_join(const PromptArgs a, const Schedule sc) {
  dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * 8ll + (threadIdx.x >> 5), id = w / (2 * kTile);
  const int r = static_cast<int>(w % (2 * kTile)), row = r % kTile;
  if (id >= sc.n_items || row >= sc.tpt * a.G) return;
  const Item x = whole_item(a, sc, id);
  const int tok = r / kTile * sc.tpt + row / a.G;
  if (tok >= x.n_tok) return;
  const int64_t part0 = id * sc.n_split;
  float2 ml[kMaxSplit / 32];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int u = 0; u < kMaxSplit / 32; ++u) {
    const int s = u * 32 + lane;
    ml[u] = make_float2(-INFINITY, 0.f);
    if (s < sc.n_split) ml[u] = sc.ml[(part0 + s) * (2 * kTile) + r];
    m = fmaxf(m, ml[u].x);
  }
  const int head = x.head * a.G + row % a.G;
  for (int i = 16; i > 0; i >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
  const float mz = m == -INFINITY ? 0.f : m;
  float o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll
  for (int u = 0; u < kMaxSplit / 32; ++u) {
    const float f = ex2(ml[u].x - mz);
    if (ml[u].y != 0.f) l += ml[u].y * f;
    for (uint32_t some = __ballot_sync(0xffffffffu, ml[u].y != 0.f); some; some &= some - 1) {
      const int s = __ffs(some) - 1;
      const float fs = __shfl_sync(0xffffffffu, f, s);
      const float* from = sc.o + ((part0 + u * 32 + s) * (2 * kTile) + r) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(from[i * 32 + lane], fs, o[i]);
    }
  }
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  const int64_t at = static_cast<int64_t>(x.qtok + tok) * a.Hq + head;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const __nv_bfloat16 b = __float2bfloat16_rn(o[i] * inv);
    a.out[at * D + i * 32 + lane] = *reinterpret_cast<const uint16_t*>(&b);
  }
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Blocks that sequences of total_q queries can take: each starts at slot
// cu_q[b] / qb + b, so the last one ends by total_q / qb, rounded up, + n_seqs - 1.
int64_t slots_of(int64_t total_q, int64_t n_seqs, int64_t qb) { return (total_q + qb - 1) / qb + n_seqs - 1; }

// Parts of an item, by the time that the sequences' average lengths suggest, in
// key tiles (1.75 us at D = 128): the rounds of CTAs that the items take, or the
// longest item, with 6 tiles to begin and end an item, 2 for the second launch
// and what the parts' outputs take to write and read.  A part has at least 512
// keys, and the parts' workspace ends at four parts an SM (78 MB).  Divided only
// where a tenth is gained: 32 heads on 8 behind 65536 keys, 256 queries 938 ->
// 256 us, 600 queries 942 -> 612, 1200 queries (152 items) 1925 -> 1305.
int parts_of(int64_t n_slots, int64_t total_q, int64_t total_k, int64_t n_seqs, int64_t n_kv_heads) {
  const int64_t sms = device_sms();
  if (n_seqs <= 0 || n_slots <= 0 || total_k / n_seqs < 1024) return 1;
  const double keys = static_cast<double>(total_k) / n_seqs, queries = static_cast<double>(total_q) / n_seqs;
  const double longest = keys / kTile, mean = fmax(keys - queries / 2, keys / 2) / kTile;
  // half of the sequences' last blocks are taken to be there
  const int64_t items = (n_slots - (n_seqs - 1) / 2) * n_kv_heads;
  auto cost = [&](int64_t s) {
    const int64_t rounds = (items * s + sms - 1) / sms;
    return fmax(longest, rounds * mean) / s + 6 * rounds + (s > 1 ? 2 + 3.0 * items * s / sms : 0);
  };
  int64_t best = 1;
  for (int64_t s = 2; s <= kMaxSplit && s * 512 <= keys && s * n_slots * n_kv_heads <= 4 * sms; ++s)
    if (cost(s) < cost(best)) best = s;
  return cost(best) < 0.9 * cost(1) ? static_cast<int>(best) : 1;
}
int64_t part_bytes(int64_t n_items, int n_split, int D) {
  return n_split == 1 ? 0 : n_items * n_split * 2 * kTile * (8 + 4ll * D);
}

// Tensor map of [tokens, heads, D] bf16 with a box of 64 elements x
// box_heads x box_tokens, 128-byte swizzle; out-of-range rows read 0.
bool map_rows(CUtensorMap* m, const void* p, int64_t tokens, int heads, int D, int64_t tok_stride, int64_t head_stride,
              int box_heads, int box_tokens) {
  static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  if (!enc) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return false;
    enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  // a dimension of one element never moves by its stride
  if (heads == 1) head_stride = D;
  if (tokens == 1) tok_stride = static_cast<int64_t>(heads) * D;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(tok_stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kSplit>
cudaError_t launch_prompt(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptArgs& a,
                          const Schedule& sc, cudaStream_t st) {
  static ReadyOnce ready;
  cudaError_t e = ready.shared_memory(k_prompt_tc<D, kSplit>, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  e = launch_after(k_prompt_tc<D, kSplit>, dim3(static_cast<unsigned>(sc.n_items * sc.n_split)), dim3(kThreads),
                   Smem<D>::kBytes, st, mq, mk, mv, a, sc);
  if (e != cudaSuccess || !kSplit) return e;
  return launch_after(k_prompt_join<D>, dim3(static_cast<unsigned>(sc.n_items * (2 * kTile / 8))), dim3(256), 0, st, a, sc);
}
template <int D>
cudaError_t launch_prompt(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptArgs& a,
                          const Schedule& sc, cudaStream_t st) {
  return sc.n_split > 1 ? launch_prompt<D, true>(mq, mk, mv, a, sc, st) : launch_prompt<D, false>(mq, mk, mv, a, sc, st);
}

}  // namespace
}  // namespace aiidx

extern "C" int ai_attend_prompt_workspace(int32_t n_seqs, int32_t total_q, int32_t total_k, int32_t n_heads,
                                          int32_t n_kv_heads, int32_t head_dim, int64_t* bytes_out) {
  using namespace aiidx;
  if (!bytes_out || n_seqs < 0 || total_q < 0 || total_k < 0 || n_heads <= 0 || n_kv_heads <= 0 ||
      n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > kTile || head_dim <= 0)
    return fail(AI_ERR_ARG, "bad sizes or null output");
  const int64_t slots = slots_of(total_q, n_seqs, 2 * (kTile / (n_heads / n_kv_heads)));
  *bytes_out = part_bytes(slots * n_kv_heads, parts_of(slots, total_q, total_k, n_seqs, n_kv_heads), head_dim);
  return AI_OK;
}

extern "C" int ai_attend_prompt(const void* q_dev, const int64_t* q_strides, const void* k_dev,
                                const int64_t* k_strides, const void* v_dev, const int64_t* v_strides,
                                const int32_t* cu_q_dev, const int32_t* cu_k_dev, int32_t n_seqs, int32_t total_q,
                                int32_t total_k, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale,
                                void* out_dev, float* lse_dev, int32_t* status_dev, void* workspace_dev,
                                int64_t workspace_bytes, void* cuda_stream) {
  using namespace aiidx;
  if (!q_strides || !k_strides || !v_strides || !cu_q_dev || !cu_k_dev) return fail(AI_ERR_ARG, "null pointer argument");
  if (n_seqs < 0 || total_q < 0 || total_k < 0) return fail(AI_ERR_ARG, "negative sequence or token count");
  // the end of the last tile behind the last token stays below 2^31
  if (total_q > kMaxTokens || total_k > kMaxTokens) return fail(AI_ERR_ARG, "more than 2^31 - 257 tokens");
  if ((total_q > 0 && (!q_dev || !out_dev)) || (total_k > 0 && (!k_dev || !v_dev)))
    return fail(AI_ERR_ARG, "null pointer argument");
  if (head_dim != 64 && head_dim != 128) return fail(AI_ERR_ARG, "head_dim must be 64 or 128");
  if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0)
    return fail(AI_ERR_ARG, "query heads must be a multiple of the key heads");
  if (n_heads / n_kv_heads > 128) return fail(AI_ERR_ARG, "more than 128 query heads per key head");
  if (!(scale >= 0.f) || scale - scale != 0.f) return fail(AI_ERR_ARG, "scale must be finite and not negative");
  if ((reinterpret_cast<uintptr_t>(q_dev) | reinterpret_cast<uintptr_t>(k_dev) | reinterpret_cast<uintptr_t>(v_dev) |
       reinterpret_cast<uintptr_t>(out_dev)) % 16 != 0)
    return fail(AI_ERR_ARG, "q, k, v and out must be 16-byte aligned");
  const struct {
    const int64_t* s;
    int64_t n[2];
  } views[3] = {{q_strides, {total_q, n_heads}}, {k_strides, {total_k, n_kv_heads}}, {v_strides, {total_k, n_kv_heads}}};
  for (const auto& x : views)
    for (int i = 0; i < 2; ++i)
      if (x.n[i] > 1 && (x.s[i] <= 0 || x.s[i] % 8 != 0 || x.s[i] > (int64_t(1) << 38)))
        return fail(AI_ERR_ARG, "token and head strides must be positive multiples of 8 elements, at most 2^38");
  if (n_seqs == 0 || total_q == 0) return AI_OK;
  PromptArgs a{};
  a.q = static_cast<const uint16_t*>(q_dev);
  a.k = static_cast<const uint16_t*>(k_dev);
  a.v = static_cast<const uint16_t*>(v_dev);
  a.q_tok = q_strides[0];
  a.q_head = q_strides[1];
  a.k_tok = k_strides[0];
  a.k_head = k_strides[1];
  a.v_tok = v_strides[0];
  a.v_head = v_strides[1];
  a.cu_q = cu_q_dev;
  a.cu_k = cu_k_dev;
  a.n_seqs = n_seqs;
  a.total_q = total_q;
  a.total_k = total_k;
  a.Hq = n_heads;
  a.Hkv = n_kv_heads;
  a.G = n_heads / n_kv_heads;
  // scale 0 weighs all keys alike; a masked score, -inf, stays -inf
  a.c2 = scale == 0.f ? 1e-30f : scale * kLog2e;
  a.out = static_cast<uint16_t*>(out_dev);
  a.lse = lse_dev;
  Schedule sc;
  sc.tpt = kTile / a.G;
  sc.qb = 2 * sc.tpt;
  const int64_t slots = slots_of(total_q, n_seqs, sc.qb);
  if (slots > 0x7fffffff) return fail(AI_ERR_ARG, "too many query blocks");
  sc.n_slots = static_cast<int>(slots);
  sc.n_items = slots * n_kv_heads;
  if (sc.n_items > 0x7fffffff) return fail(AI_ERR_ARG, "too many query blocks");
  sc.n_split = parts_of(slots, total_q, total_k, n_seqs, n_kv_heads);
  sc.ml = nullptr;
  sc.o = nullptr;
  if (sc.n_split > 1) {
    if (!workspace_dev || reinterpret_cast<uintptr_t>(workspace_dev) % 16 != 0 ||
        workspace_bytes < part_bytes(sc.n_items, sc.n_split, head_dim))
      return fail(AI_ERR_ARG, "workspace too small or not 16-byte aligned");
    const int64_t parts = sc.n_items * sc.n_split;
    sc.o = static_cast<float*>(workspace_dev);
    sc.ml = reinterpret_cast<float2*>(sc.o + parts * 2 * kTile * head_dim);
  }
  a.status = status_dev ? status_dev : default_status();
  if (!a.status) return fail(AI_ERR_CUDA, "the device's status word was not found");
  CUtensorMap mq, mk, mv;
  // without keys nothing is loaded, but a map needs a row
  const bool none = total_k == 0;
  if (!map_rows(&mq, q_dev, total_q, n_heads, head_dim, a.q_tok, a.q_head, a.G, sc.tpt) ||
      !map_rows(&mk, none ? q_dev : k_dev, none ? 1 : total_k, n_kv_heads, head_dim, a.k_tok, none ? head_dim : a.k_head,
                1, kTile) ||
      !map_rows(&mv, none ? q_dev : v_dev, none ? 1 : total_k, n_kv_heads, head_dim, a.v_tok, none ? head_dim : a.v_head,
                1, kTile))
    return fail(AI_ERR_CUDA, "tensor map encoding failed");
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e =
      head_dim == 64 ? launch_prompt<64>(mq, mk, mv, a, sc, st) : launch_prompt<128>(mq, mk, mv, a, sc, st);
  return e == cudaSuccess ? AI_OK : fail(AI_ERR_CUDA, cudaGetErrorString(e));
}
