// Attention of single rows over a paged key-value cache:
//   cached    row r reads tokens 0 .. len - 1 of its sequence (decode);
//   selected  row t reads the tokens ids[t, :] that the index selected.
//
//   s_j = scale * q . k_j,   o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
//   m = max_j s_j,           lse = m + ln sum_j e^(s_j - m)
//
// in one pass over the keys, with m, the sum and o kept in fp32 registers
// (base-2 exponents: scale * log2 e is one factor).  The G = Hq / Hkv query
// heads that share a key head are the rows of one matrix product, so every
// key and value is read once per group.  What bounds it is reading the keys
// and values; the products are mma.sync m16n8k16 (at G <= 64 rows a 128-row
// tcgen05 tile would be half empty or worse, and its operands would have to
// be converted and rearranged by extra warps: the fp8 codes are widened in
// registers here).
//
// Work: tiles of 64 keys.  The CTAs (two per SM) divide all tiles of the
// batch evenly, whatever the lengths; a row whose tiles lie in several CTAs
// is joined by a second kernel from per-CTA partial results, always in tile
// order (no atomics: results do not depend on timing).  With several rows
// per CTA (prefill) whole rows are dealt out in turn, heads outermost, so
// that rows running at the same time read the same head's keys (L2), and
// only the last part wave is divided.
#include <cmath>

#include "../../include/ai_index.h"
#include "common.cuh"
#include "kernels.h"

namespace aiidx {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct RowsArgs {
  const uint16_t* q;        // [R, Hq, D] bf16
  const uint8_t* k;         // pages of one layer, bytes
  const uint8_t* v;
  const float* ks;          // [n_pages * page_size, Hkv] or nullptr
  const float* vs;
  const int32_t* tables;    // [n_seqs, width]
  const int32_t* lens;      // [n_seqs]
  const int32_t* seqs;      // [R] or nullptr
  int seq_mul;              // sequence of row r without seqs: r * seq_mul
  const int32_t* ids;       // [R, n_ids] or nullptr (cached)
  int R, n_ids, Hq, Hkv, G;
  int n_mb, mb_rows;        // row blocks per key head, query heads per block
  int n_seqs, width, n_pages, page_size;
  float c2;                 // scale * log2 e
  uint16_t* out;            // [R, Hq, D] bf16
  float* lse;               // [R, Hq] or nullptr
  float* part;              // partial results: [2 * grid][16 MT][D + 2]
  int32_t* meta;            // [grid][4]
  int32_t* status;          // or nullptr
};

// ------------------------------------------------------------- warp products
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// Two e4m3 codes (low byte first) to two bf16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint16_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(codes, __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x, f.y);
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes to shared memory, zeros where !real.
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4z(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

// ------------------------------------------------------------ shared memory
// What the consumer of a tile has to know about it.
struct TileMeta {
  int row, head;   // row of q; key head * n_mb + row block
  int first, last; // of this CTA's share of the row
  int slot;        // -1: the row lies whole in this CTA; 0 / 1: partial result slot
  int any;         // some key of the tile is real
};

template <int D, bool FP8, int MT>
struct Layout {
  static constexpr int kRow = FP8 ? D : 2 * D;          // bytes of a key row
  static constexpr int kChunks = kRow / 16;
  static constexpr int kKV = kTile * kRow;              // bytes of a K or V tile
  static constexpr int kQRow = 2 * D + 16;              // padded: rows fall on different banks
  static constexpr int kQ = 16 * MT * kQRow;
  static constexpr int kScales = FP8 ? 2 * kTile * 4 : 0;
  static constexpr int kStage = 2 * kKV + kQ + kScales;
  static constexpr int kWK = 4 / MT;                    // warps along the keys
  static constexpr int kMerge = (kWK - 1) * 16 * MT * (D + 2) * 4;
  static constexpr int kStages = FP8 ? (MT == 1 ? 4 : 3) : 2;
  static constexpr int kRing = kStages + 1;
  static constexpr int kBytes =
      kStages * kStage + kMerge + kRing * (kTile * 4 + static_cast<int>(sizeof(TileMeta)));
  // 16-byte chunk c of tile row r is stored at chunk c ^ swz(r), so that the
  // eight rows of an ldmatrix, and (fp8) the two rows of a quarter warp's
  // 16-byte loads, fall on different banks
  __device__ static int swz(int r) {
    if constexpr (!FP8) return r & 7;
    if constexpr (kChunks == 8) return ((r & 1) << 2) | ((r >> 1) & 3);
    return (r >> 1) & 3;
  }
};

// ----------------------------------------------------------- division of work
// Item: one row and one (key head, row block).  Tiles of an item are
// consecutive; CTA c takes the whole items it, it + grid, .. < n_whole and
// then the tiles [b0, b1) of the items from n_whole on.
struct Walk {
  int it;             // whole items: the current one
  int n_whole, grid;
  int64_t b, b1;      // divided tiles: current, end
  int row, head, tile, n_tiles;  // current position
  bool divided;
};

__device__ __forceinline__ int seq_of(const RowsArgs& a, int row) {
  return a.seqs ? a.seqs[row] : row * a.seq_mul;
}
__device__ __forceinline__ int len_of(const RowsArgs& a, int row) {
  const int s = seq_of(a, row);
  if (s < 0 || s >= a.n_seqs) return 0;
  const int64_t most = static_cast<int64_t>(a.width) * a.page_size;
  const int n = a.lens[s];
  if ((n < 0 || n > most) && a.status) atomicOr(a.status, AI_DEVFLAG_RANGE);
  return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}
__device__ __forceinline__ int tiles_of(const RowsArgs& a, int row) {
  return ((a.ids ? a.n_ids : len_of(a, row)) + kTile - 1) / kTile;
}

// Block-wide sum and exclusive prefix of one int64 per thread.
__device__ int64_t block_scan(int64_t x, int64_t* total, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int64_t before = 0, sum = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sums[w];
    sum += warp_sums[w];
  }
  *total = sum;
  return before + inc - x;
}

template <int D, bool FP8, int MT>
__global__ void __launch_bounds__(kThreads, 2) k_attend_rows(const RowsArgs a) {
  using L = Layout<D, FP8, MT>;
  constexpr int S = L::kStages;
  constexpr int WK = L::kWK;
  constexpr int NK = kTile / WK;   // keys of a tile per warp
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* merge = smem + S * L::kStage;
  int32_t* ring_row = reinterpret_cast<int32_t*>(merge + L::kMerge);
  TileMeta* ring_meta = reinterpret_cast<TileMeta*>(ring_row + L::kRing * kTile);
  __shared__ int64_t sh_scan[kThreads / 32];
  __shared__ int64_t sh_b0;
  __shared__ int sh_row;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int wm = warp % MT, wk = warp / MT;
  const int n_heads = a.Hkv * a.n_mb;
  const int grid = gridDim.x, cta = blockIdx.x;

  // ---------------------------------------------------- this CTA's share
  Walk w;
  w.grid = grid;
  w.it = cta;
  w.n_whole = 0;
  int start_tile = 0;     // first divided tile within its row's tiles of all heads
  int64_t total;
  if (a.ids) {
    const int64_t items = static_cast<int64_t>(a.R) * n_heads;
    const int nt = (a.n_ids + kTile - 1) / kTile;
    w.n_whole = static_cast<int>(items / grid) * grid;
    total = (items - w.n_whole) * nt;
    w.b = total * cta / grid;
    w.b1 = total * (cta + 1) / grid;
  } else {
    // two passes over the lengths: the number of tiles, and the row where
    // this CTA's share begins
    total = 0;
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
      int64_t sum;
      const int r = r0 + tid;
      block_scan(r < a.R ? tiles_of(a, r) : 0, &sum, sh_scan);
      total += sum;
    }
    total *= n_heads;
    w.b = total * cta / grid;
    w.b1 = total * (cta + 1) / grid;
    int64_t seen = 0;
    for (int r0 = 0; r0 < a.R; r0 += kThreads) {
      int64_t sum;
      const int r = r0 + tid;
      const int64_t n = r < a.R ? static_cast<int64_t>(tiles_of(a, r)) * n_heads : 0;
      const int64_t p = seen + block_scan(n, &sum, sh_scan);
      if (n > 0 && p <= w.b && w.b < p + n) {
        sh_row = r;
        sh_b0 = p;
      }
      seen += sum;
      // rows that see nothing: zeros, and the log of an empty sum
      for (int rr = r0; rr < r0 + kThreads && rr < a.R; ++rr) {
        if (rr % grid != cta || tiles_of(a, rr) > 0) continue;
        for (int i = tid; i < a.Hq * D / 2; i += kThreads)
          reinterpret_cast<uint32_t*>(a.out)[static_cast<int64_t>(rr) * a.Hq * D / 2 + i] = 0;
        if (a.lse)
          for (int i = tid; i < a.Hq; i += kThreads) a.lse[static_cast<int64_t>(rr) * a.Hq + i] = -INFINITY;
        if (a.status && tid == 0) {
          const int s = seq_of(a, rr);
          if (s < 0 || s >= a.n_seqs) atomicOr(a.status, AI_DEVFLAG_RANGE);
        }
      }
    }
    __syncthreads();
    if (w.b < w.b1) {
      w.row = sh_row;
      start_tile = static_cast<int>(w.b - sh_b0);
    }
  }
  // position the walk on its first tile
  w.divided = w.it >= w.n_whole;
  auto locate_item = [&](int64_t item) {   // selected: heads outermost
    w.head = static_cast<int>(item / a.R);
    w.row = static_cast<int>(item % a.R);
  };
  auto enter_divided = [&]() {
    w.divided = true;
    if (a.ids) {
      w.n_tiles = (a.n_ids + kTile - 1) / kTile;
      locate_item(w.n_whole + w.b / w.n_tiles);
      w.tile = static_cast<int>(w.b % w.n_tiles);
    } else if (w.b < w.b1) {
      w.n_tiles = tiles_of(a, w.row);
      w.head = start_tile / w.n_tiles;
      w.tile = start_tile % w.n_tiles;
    }
  };
  if (w.divided) {
    enter_divided();
  } else {
    locate_item(w.it);
    w.n_tiles = (a.n_ids + kTile - 1) / kTile;
    w.tile = 0;
  }
  const int64_t n_mine =
      (w.n_whole > 0 ? static_cast<int64_t>(w.n_whole / grid) * ((a.n_ids + kTile - 1) / kTile) : 0) + (w.b1 - w.b);
  const int64_t b_begin = w.b;

  // what the joining kernel reads: the item that began before this CTA, or
  // -1 (0), whether it ends here (1), and the item that begins here and goes
  // on in the next CTA that has a share, or -1 (2)
  if (tid == 0) {
    a.meta[cta * 4 + 0] = -1;
    a.meta[cta * 4 + 1] = 1;
    a.meta[cta * 4 + 2] = -1;
    a.meta[cta * 4 + 3] = -1;
  }
  // the slot of the current item's share, -1 where the item lies whole here
  auto slot_of = [&]() {
    if (!w.divided) return -1;
    const int64_t i0 = w.b - w.tile, i1 = i0 + w.n_tiles;
    if (i0 < b_begin) return i1 > w.b1 ? 2 : 0;   // 2: began before and goes on
    return i1 > w.b1 ? 1 : -1;
  };
  auto advance = [&]() {
    ++w.tile;
    if (w.divided) ++w.b;
    if (w.tile < w.n_tiles) return;
    w.tile = 0;
    if (!w.divided) {
      w.it += grid;
      if (w.it >= w.n_whole) enter_divided();
      else locate_item(w.it);
    } else if (a.ids) {
      if (++w.row == a.R) {
        w.row = 0;
        ++w.head;
      }
    } else if (++w.head == n_heads) {
      w.head = 0;
      if (w.b < w.b1) {
        do ++w.row;
        while (w.row < a.R && tiles_of(a, w.row) == 0);
        w.n_tiles = w.row < a.R ? tiles_of(a, w.row) : 1;
      }
    }
  };

  // ------------------------------------------------- plan, two steps ahead
  // Threads 0..63 follow the walk; thread i looks up key i of a tile.
  int plan_tok = -1;               // token of the tile planned next
  TileMeta plan_meta{};
  int plan_seq = 0;
  auto plan_token = [&](int64_t n) {  // step 1: the token
    plan_tok = -1;
    if (n >= n_mine) return;
    const int s = seq_of(a, w.row);
    const int len = len_of(a, w.row);
    const int at = w.tile * kTile + tid;
    int tok = -1;
    if (a.ids) {
      if (at < a.n_ids) {
        tok = a.ids[static_cast<int64_t>(w.row) * a.n_ids + at];
        if (tok >= len) {
          if (a.status) atomicOr(a.status, AI_DEVFLAG_RANGE);
          tok = -1;
        }
      }
    } else if (at < len) {
      tok = at;
    }
    plan_tok = tok < 0 ? -1 : tok;
    plan_seq = s;
    plan_meta.row = w.row;
    plan_meta.head = w.head;
    int slot = slot_of();
    plan_meta.first = w.tile == 0 || (w.divided && w.b == b_begin);
    plan_meta.last = w.tile == w.n_tiles - 1 || (w.divided && w.b == w.b1 - 1);
    if (tid == 0 && plan_meta.first && slot >= 0) {
      const int item = w.row * n_heads + w.head;
      if (slot == 1) a.meta[cta * 4 + 2] = item;
      else {
        a.meta[cta * 4 + 0] = item;
        a.meta[cta * 4 + 1] = slot == 0;
      }
    }
    plan_meta.slot = slot == 2 ? 0 : slot;
    advance();
  };
  int plan_row = -1;
  auto plan_lookup = [&]() {          // step 2: its page
    plan_row = -1;
    if (plan_tok >= 0) {
      const int page = a.tables[static_cast<int64_t>(plan_seq) * a.width + plan_tok / a.page_size];
      if (page >= 0 && page < a.n_pages) plan_row = page * a.page_size + plan_tok % a.page_size;
      else if (a.status) atomicOr(a.status, AI_DEVFLAG_RANGE);
    }
  };
  auto plan_store = [&](int64_t n, int row, TileMeta m) {
    const int e = static_cast<int>(n % L::kRing);
    ring_row[e * kTile + tid] = row;
    if (tid == 0) {
      m.any = 0;
      ring_meta[e] = m;
    }
  };

  auto issue = [&](int64_t n) {
    if (n < n_mine) {
      const int e = static_cast<int>(n % L::kRing);
      const TileMeta m = ring_meta[e];
      const uint32_t st = smem_u32(smem + (n % S) * L::kStage);
      const int h = m.head / a.n_mb;
      const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * L::kRow;
      const int c = tid % L::kChunks;
      for (int r = tid / L::kChunks; r < kTile; r += kThreads / L::kChunks) {
        const int row = ring_row[e * kTile + r];
        const int64_t off = row < 0 ? 0 : row * row_bytes + h * L::kRow + c * 16;
        const uint32_t dst = st + r * L::kRow + ((c ^ L::swz(r)) << 4);
        cp16z(dst, a.k + off, row >= 0);
        cp16z(dst + L::kKV, a.v + off, row >= 0);
      }
      if constexpr (FP8) {
        const int r = tid & 63;
        const int row = ring_row[e * kTile + r];
        const float* src = tid < 64 ? a.ks : a.vs;
        const int64_t off = row < 0 ? 0 : static_cast<int64_t>(row) * a.Hkv + h;
        cp4z(st + 2 * L::kKV + L::kQ + tid * 4, src + off, row >= 0);
      }
      if (m.first) {
        const int h0 = h * a.G + (m.head % a.n_mb) * a.mb_rows;
        const int n_rows = min(a.mb_rows, (h + 1) * a.G - h0);
        for (int i = tid; i < 16 * MT * (D / 8); i += kThreads) {
          const int r = i / (D / 8), cc = i % (D / 8);
          const bool real = r < n_rows;
          const uint16_t* src = a.q + (static_cast<int64_t>(m.row) * a.Hq + h0 + (real ? r : 0)) * D + cc * 8;
          cp16z(st + 2 * L::kKV + r * L::kQRow + cc * 16, src, real);
        }
      }
    }
    cp_async_commit();
  };

  // -------------------------------------------------------------- prologue
  if (warp < 2) {
    for (int n = 0; n < S; ++n) {
      plan_token(n);
      plan_lookup();
      plan_store(n, plan_row, plan_meta);
    }
    plan_token(S);
  }
  __syncthreads();
  for (int n = 0; n < S - 1; ++n) issue(n);

  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m_run[2], l_run[2];

  // ------------------------------------------------------------- main loop
  for (int64_t n = 0; n < n_mine; ++n) {
    cp_async_wait<S - 2>();
    __syncthreads();
    issue(n + S - 1);
    TileMeta next_meta;
    if (warp < 2) {
      plan_lookup();                 // tile n + S
      next_meta = plan_meta;
    }
    const int next_row = plan_row;
    if (warp < 2) plan_token(n + S + 1);

    const int e = static_cast<int>(n % L::kRing);
    const TileMeta m = ring_meta[e];
    const uint8_t* stage = smem + (n % S) * L::kStage;
    const uint32_t sk = smem_u32(stage);
    const uint32_t sv = sk + L::kKV;
    if (m.first) {
      const uint8_t* sq = stage + 2 * L::kKV + wm * 16 * L::kQRow;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if constexpr (!FP8) {
          ldsm4(qf[kk], smem_u32(sq) + (lane & 15) * L::kQRow + kk * 32 + (lane >> 4) * 16);
        } else {
          // the product's sum over d in the order of the codes' 16-byte loads
          const int d = (kk / 4) * 64 + t * 16 + (kk % 4) * 4;
          const uint2 x = *reinterpret_cast<const uint2*>(sq + g * L::kQRow + d * 2);
          const uint2 y = *reinterpret_cast<const uint2*>(sq + (g + 8) * L::kQRow + d * 2);
          qf[kk][0] = x.x;
          qf[kk][1] = y.x;
          qf[kk][2] = x.y;
          qf[kk][3] = y.y;
        }
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m_run[0] = m_run[1] = -INFINITY;
      l_run[0] = l_run[1] = 0.f;
    }
    const int32_t* rows = ring_row + e * kTile + wk * NK;
    bool any = false;
#pragma unroll
    for (int i = 0; i < NK; i += 32) any |= (i + lane < NK) && rows[i + lane] >= 0;
    if (__any_sync(0xffffffffu, any)) {
      float s[NK / 8][4];
#pragma unroll
      for (int j = 0; j < NK / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      if constexpr (!FP8) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
          for (int j = 0; j < NK / 16; ++j) {
            uint32_t b[4];
            const int r = wk * NK + j * 16 + (lane & 7) + ((lane >> 4) << 3);
            const int c = kk * 2 + ((lane >> 3) & 1);
            ldsm4(b, sk + r * L::kRow + ((c ^ L::swz(r)) << 4));
            mma_bf16(s[2 * j], qf[kk], b[0], b[1]);
            mma_bf16(s[2 * j + 1], qf[kk], b[2], b[3]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NK / 8; ++j) {
          const int r = wk * NK + j * 8 + g;
#pragma unroll
          for (int c4 = 0; c4 < D / 64; ++c4) {
            const uint4 x = *reinterpret_cast<const uint4*>(stage + r * L::kRow + (((c4 * 4 + t) ^ L::swz(r)) << 4));
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16(s[j], qf[c4 * 4 + i], e4m3x2_to_bf16x2(static_cast<uint16_t>(u[i] & 0xffff)),
                       e4m3x2_to_bf16x2(static_cast<uint16_t>(u[i] >> 16)));
          }
        }
      }
      // scale, mask and the running maximum
      const float* ksc = reinterpret_cast<const float*>(stage + 2 * L::kKV + L::kQ) + wk * NK;
      float mx[2] = {m_run[0], m_run[1]};
#pragma unroll
      for (int j = 0; j < NK / 8; ++j) {
        const int2 rr = *reinterpret_cast<const int2*>(rows + j * 8 + 2 * t);
        float f0 = a.c2, f1 = a.c2;
        if constexpr (FP8) {
          f0 *= ksc[j * 8 + 2 * t];
          f1 *= ksc[j * 8 + 2 * t + 1];
        }
        s[j][0] = rr.x >= 0 ? s[j][0] * f0 : -INFINITY;
        s[j][1] = rr.y >= 0 ? s[j][1] * f1 : -INFINITY;
        s[j][2] = rr.x >= 0 ? s[j][2] * f0 : -INFINITY;
        s[j][3] = rr.y >= 0 ? s[j][3] * f1 : -INFINITY;
        mx[0] = fmaxf(mx[0], fmaxf(s[j][0], s[j][1]));
        mx[1] = fmaxf(mx[1], fmaxf(s[j][2], s[j][3]));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
      }
      // a row without a finite score so far: exponents against 0 (all e^-inf = 0)
      const float mu[2] = {mx[0] == -INFINITY ? 0.f : mx[0], mx[1] == -INFINITY ? 0.f : mx[1]};
      const float al[2] = {exp2_approx(m_run[0] - mu[0]), exp2_approx(m_run[1] - mu[1])};
      const bool moved = mx[0] != m_run[0] || mx[1] != m_run[1];
      m_run[0] = mx[0];
      m_run[1] = mx[1];
      if (__any_sync(0xffffffffu, moved)) {
        l_run[0] *= al[0];
        l_run[1] *= al[1];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= al[0];
          o[i][1] *= al[0];
          o[i][2] *= al[1];
          o[i][3] *= al[1];
        }
      }
      // the weights, rounded once to bf16 for the product with v; their sum
      // is taken before that rounding
      uint32_t p[NK / 16][4];
#pragma unroll
      for (int j = 0; j < NK / 8; ++j) {
        const float e0 = exp2_approx(s[j][0] - mu[0]), e1 = exp2_approx(s[j][1] - mu[0]);
        const float e2 = exp2_approx(s[j][2] - mu[1]), e3 = exp2_approx(s[j][3] - mu[1]);
        l_run[0] += e0 + e1;
        l_run[1] += e2 + e3;
        float f0 = 1.f, f1 = 1.f;
        if constexpr (FP8) {
          f0 = ksc[kTile + j * 8 + 2 * t];
          f1 = ksc[kTile + j * 8 + 2 * t + 1];
        }
        p[j / 2][(j & 1) * 2 + 0] = pack_bf16(e0 * f0, e1 * f1);
        p[j / 2][(j & 1) * 2 + 1] = pack_bf16(e2 * f0, e3 * f1);
      }
      if constexpr (!FP8) {
#pragma unroll
        for (int j = 0; j < NK / 16; ++j) {
#pragma unroll
          for (int dd = 0; dd < D / 16; ++dd) {
            uint32_t b[4];
            const int r = wk * NK + j * 16 + (lane & 15);
            const int c = dd * 2 + (lane >> 4);
            ldsm4t(b, sv + r * L::kRow + ((c ^ L::swz(r)) << 4));
            mma_bf16(o[2 * dd], p[j], b[0], b[1]);
            mma_bf16(o[2 * dd + 1], p[j], b[2], b[3]);
          }
        }
      } else {
        // 16-bit transposed loads bring two neighbouring codes of two keys;
        // accumulator 2 i holds the even, 2 i + 1 the odd d of 16-code chunk i
#pragma unroll
        for (int j = 0; j < NK / 16; ++j) {
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t b[4];
            const int r = wk * NK + j * 16 + (lane & 15);
            const int c = cc * 2 + (lane >> 4);
            ldsm4t(b, sv + r * L::kRow + ((c ^ L::swz(r)) << 4));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t lo = b[2 * i], hi = b[2 * i + 1];
              mma_bf16(o[(cc * 2 + i) * 2], p[j],
                       e4m3x2_to_bf16x2(static_cast<uint16_t>(__byte_perm(lo, 0, 0x4420))),
                       e4m3x2_to_bf16x2(static_cast<uint16_t>(__byte_perm(hi, 0, 0x4420))));
              mma_bf16(o[(cc * 2 + i) * 2 + 1], p[j],
                       e4m3x2_to_bf16x2(static_cast<uint16_t>(__byte_perm(lo, 0, 0x4431))),
                       e4m3x2_to_bf16x2(static_cast<uint16_t>(__byte_perm(hi, 0, 0x4431))));
            }
          }
        }
      }
    }
    if (warp < 2) plan_store(n + S, next_row, next_meta);

    if (m.last) {
      // the row sums over the four lanes of a row, then over the key warps
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
        l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
      }
      float* mine = reinterpret_cast<float*>(merge) + static_cast<int64_t>((wk - 1) * MT + wm) * 16 * (D + 2);
      if constexpr (WK > 1) {
        if (wk > 0) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            *reinterpret_cast<float2*>(mine + g * (D + 2) + i * 8 + 2 * t) = make_float2(o[i][0], o[i][1]);
            *reinterpret_cast<float2*>(mine + (g + 8) * (D + 2) + i * 8 + 2 * t) = make_float2(o[i][2], o[i][3]);
          }
          if (t == 0) {
            *reinterpret_cast<float2*>(mine + g * (D + 2) + D) = make_float2(m_run[0], l_run[0]);
            *reinterpret_cast<float2*>(mine + (g + 8) * (D + 2) + D) = make_float2(m_run[1], l_run[1]);
          }
        }
        __syncthreads();
        if (wk == 0) {
          for (int ww = 1; ww < WK; ++ww) {
            const float* src = reinterpret_cast<const float*>(merge) + static_cast<int64_t>((ww - 1) * MT + wm) * 16 * (D + 2);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float* sr = src + (g + half * 8) * (D + 2);
              const float2 ml = *reinterpret_cast<const float2*>(sr + D);
              const float mn = fmaxf(m_run[half], ml.x);
              const float mz = mn == -INFINITY ? 0.f : mn;
              const float f0 = exp2_approx(m_run[half] - mz), f1 = exp2_approx(ml.x - mz);
              m_run[half] = mn;
              l_run[half] = l_run[half] * f0 + ml.y * f1;
#pragma unroll
              for (int i = 0; i < D / 8; ++i) {
                const float2 x = *reinterpret_cast<const float2*>(sr + i * 8 + 2 * t);
                o[i][2 * half] = o[i][2 * half] * f0 + x.x * f1;
                o[i][2 * half + 1] = o[i][2 * half + 1] * f0 + x.y * f1;
              }
            }
          }
        }
      }
      if (wk == 0) {
        const int h = m.head / a.n_mb;
        const int h0 = h * a.G + (m.head % a.n_mb) * a.mb_rows;
        const int n_rows = min(a.mb_rows, (h + 1) * a.G - h0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int r = wm * 16 + g + half * 8;
          if (r >= n_rows) continue;
          // where accumulator pair i of this lane belongs (fp8: even and odd d)
          if (m.slot < 0) {
            const float inv = l_run[half] == 0.f ? 0.f : 1.f / l_run[half];
            uint16_t* dst = a.out + (static_cast<int64_t>(m.row) * a.Hq + h0 + r) * D;
            if constexpr (!FP8) {
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<uint32_t*>(dst + i * 8 + 2 * t) =
                    pack_bf16(o[i][2 * half] * inv, o[i][2 * half + 1] * inv);
            } else {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint2 x = make_uint2(pack_bf16(o[2 * i][2 * half] * inv, o[2 * i + 1][2 * half] * inv),
                                           pack_bf16(o[2 * i][2 * half + 1] * inv, o[2 * i + 1][2 * half + 1] * inv));
                *reinterpret_cast<uint2*>(dst + i * 16 + 4 * t) = x;
              }
            }
            if (a.lse && t == 0)
              a.lse[static_cast<int64_t>(m.row) * a.Hq + h0 + r] =
                  l_run[half] == 0.f ? -INFINITY : (m_run[half] + log2f(l_run[half])) * kLn2;
          } else {
            float* dst = a.part + (static_cast<int64_t>(cta * 2 + m.slot) * 16 * MT + r) * (D + 2);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              if constexpr (!FP8) {
                *reinterpret_cast<float2*>(dst + i * 8 + 2 * t) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
              } else {
                dst[(i / 2) * 16 + 4 * t + (i & 1)] = o[i][2 * half];
                dst[(i / 2) * 16 + 4 * t + 2 + (i & 1)] = o[i][2 * half + 1];
              }
            }
            if (t == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(m_run[half], l_run[half]);
          }
        }
      }
    }
  }
  cp_async_wait_all();
}

// Joins the parts of a row that begins in CTA blockIdx.x and goes on in the
// following ones; blockIdx.y is the row within the block of query heads.
template <int D>
__global__ void __launch_bounds__(D) k_join_rows(const RowsArgs a, int n_ctas, int rows_per_slot) {
  const int c = blockIdx.x, r = blockIdx.y, d = threadIdx.x;
  const int item = a.meta[c * 4 + 2];
  if (item < 0) return;
  const int n_heads = a.Hkv * a.n_mb;
  const int head = item % n_heads, row = item / n_heads;
  const int h = head / a.n_mb;
  const int h0 = h * a.G + (head % a.n_mb) * a.mb_rows;
  if (r >= min(a.mb_rows, (h + 1) * a.G - h0)) return;
  const float* p = a.part + (static_cast<int64_t>(c * 2 + 1) * rows_per_slot + r) * (D + 2);
  float m = p[D], l = p[D + 1], o = p[d];
  for (int n = c + 1; n < n_ctas; ++n) {
    if (a.meta[n * 4] < 0) continue;  // a CTA without a share
    const bool ends = a.meta[n * 4 + 1] != 0;
    const float* q = a.part + (static_cast<int64_t>(n * 2) * rows_per_slot + r) * (D + 2);
    const float mn = fmaxf(m, q[D]);
    const float mz = mn == -INFINITY ? 0.f : mn;
    const float f0 = exp2_approx(m - mz), f1 = exp2_approx(q[D] - mz);
    m = mn;
    l = l * f0 + q[D + 1] * f1;
    o = o * f0 + q[d] * f1;
    if (ends) break;
  }
  const __nv_bfloat16 b = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  a.out[(static_cast<int64_t>(row) * a.Hq + h0 + r) * D + d] = *reinterpret_cast<const uint16_t*>(&b);
  if (a.lse && d == 0)
    a.lse[static_cast<int64_t>(row) * a.Hq + h0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, bool FP8, int MT>
cudaError_t launch_mt(const RowsArgs& a, int grid, cudaStream_t st) {
  using L = Layout<D, FP8, MT>;
  static_assert(2 * (L::kBytes + 2048) <= 227 * 1024, "two CTAs per SM");
  cudaError_t e = cudaFuncSetAttribute(k_attend_rows<D, FP8, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  count_launch();
  k_attend_rows<D, FP8, MT><<<grid, kThreads, L::kBytes, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  count_launch();
  k_join_rows<D><<<dim3(grid, a.mb_rows), D, 0, st>>>(a, grid, 16 * MT);
  return cudaGetLastError();
}

template <int D, bool FP8>
cudaError_t launch_d(const RowsArgs& a, int grid, cudaStream_t st) {
  if (a.mb_rows <= 16) return launch_mt<D, FP8, 1>(a, grid, st);
  if (a.mb_rows <= 32) return launch_mt<D, FP8, 2>(a, grid, st);
  return launch_mt<D, FP8, 4>(a, grid, st);
}

int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

int num_sms() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// The largest grid (partial results are sized for it).
int max_grid() { return 2 * num_sms(); }

int64_t workspace_for(int Hq, int Hkv, int D) {
  const int G = Hq / Hkv;
  const int mb = (G + 63) / 64;
  const int rows = ((G + mb - 1) / mb + 15) / 16 * 16;
  const int padded = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
  const int64_t g = max_grid();
  return g * 16 + g * 2 * padded * (D + 2) * 4;
}

int run_rows(const ai_cache* c, int32_t layer, const void* q, int32_t R, int32_t Hq, const int32_t* ids, int32_t n_ids,
             const int32_t* seqs, float scale, void* out, float* lse, void* ws, int64_t ws_bytes, void* stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  if ((R > 0 && (!q || !out)) || !ws) return fail(AI_ERR_ARG, "null pointer argument");
  if (layer < 0 || layer >= c->n_layers) return fail(AI_ERR_ARG, "layer out of range");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(AI_ERR_ARG, "head_dim must be 64 or 128");
  if (R < 0 || Hq <= 0 || Hq % c->n_kv_heads != 0) return fail(AI_ERR_ARG, "query heads must be a multiple of the key heads");
  if (R > 0 && !seqs && c->n_seqs != R && !(ids && c->n_seqs == 1))
    return fail(AI_ERR_ARG, "without seqs the table needs one row per query row");
  if (!(scale >= 0.f) || scale - scale != 0.f) return fail(AI_ERR_ARG, "scale must be finite and not negative");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(ws)) % 16 != 0)
    return fail(AI_ERR_ARG, "q, out and the workspace must be 16-byte aligned");
  if (ws_bytes < workspace_for(Hq, c->n_kv_heads, c->head_dim)) return fail(AI_ERR_ARG, "workspace too small");
  const int G = Hq / c->n_kv_heads;
  const int n_mb = (G + 63) / 64;
  if (static_cast<int64_t>(R) * c->n_kv_heads * n_mb > 0x7fffffff) return fail(AI_ERR_ARG, "too many rows times key heads");
  if (R == 0) return AI_OK;
  RowsArgs a{};
  const int64_t tokens = static_cast<int64_t>(c->n_pages) * c->page_size;
  const int64_t elems = tokens * c->n_kv_heads * c->head_dim;
  const int es = c->dtype == AI_BF16 ? 2 : 1;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint8_t*>(c->k) + layer * elems * es;
  a.v = static_cast<const uint8_t*>(c->v) + layer * elems * es;
  if (es == 1) {
    a.ks = c->k_scale + layer * tokens * c->n_kv_heads;
    a.vs = c->v_scale + layer * tokens * c->n_kv_heads;
  }
  a.tables = c->tables;
  a.lens = c->lens;
  a.seqs = seqs;
  a.seq_mul = c->n_seqs == R ? 1 : 0;
  a.ids = ids;
  a.R = R;
  a.n_ids = n_ids;
  a.Hq = Hq;
  a.Hkv = c->n_kv_heads;
  a.G = G;
  a.n_mb = n_mb;
  a.mb_rows = (G + n_mb - 1) / n_mb;
  a.n_seqs = c->n_seqs;
  a.width = c->max_pages;
  a.n_pages = c->n_pages;
  a.page_size = c->page_size;
  a.c2 = scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = c->status;
  const int64_t most = ids ? n_ids : static_cast<int64_t>(c->max_pages) * c->page_size;
  const int64_t tiles = static_cast<int64_t>(R) * a.Hkv * n_mb * ((most + kTile - 1) / kTile);
  const int grid = static_cast<int>(tiles < 1 ? 1 : (tiles < max_grid() ? tiles : max_grid()));
  a.meta = static_cast<int32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + static_cast<int64_t>(max_grid()) * 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c->head_dim == 64) e = es == 2 ? launch_d<64, false>(a, grid, st) : launch_d<64, true>(a, grid, st);
  else e = es == 2 ? launch_d<128, false>(a, grid, st) : launch_d<128, true>(a, grid, st);
  return e == cudaSuccess ? AI_OK : fail(AI_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace
}  // namespace aiidx

extern "C" int ai_attend_workspace(int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int64_t* bytes_out) {
  using namespace aiidx;
  if (!bytes_out || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || head_dim <= 0)
    return fail(AI_ERR_ARG, "bad head counts or null output");
  *bytes_out = workspace_for(n_heads, n_kv_heads, head_dim);
  return AI_OK;
}

extern "C" int ai_attend_cached(const ai_cache* cache, int32_t layer, const void* q_dev, int32_t n_rows,
                                int32_t n_heads, const int32_t* seqs_dev, float scale, void* out_dev,
                                float* lse_dev, void* workspace_dev, int64_t workspace_bytes, void* cuda_stream) {
  return aiidx::run_rows(cache, layer, q_dev, n_rows, n_heads, nullptr, 0, seqs_dev, scale, out_dev, lse_dev,
                         workspace_dev, workspace_bytes, cuda_stream);
}

extern "C" int ai_attend_selected(const ai_cache* cache, int32_t layer, const void* q_dev, const int32_t* ids_dev,
                                  int32_t T, int32_t k, int32_t n_heads, const int32_t* seqs_dev, float scale,
                                  void* out_dev, float* lse_dev, void* workspace_dev, int64_t workspace_bytes,
                                  void* cuda_stream) {
  using namespace aiidx;
  if (!ids_dev) return fail(AI_ERR_ARG, "null pointer argument");
  if (k <= 0) return fail(AI_ERR_ARG, "k must be positive");
  return run_rows(cache, layer, q_dev, T, n_heads, ids_dev, k, seqs_dev, scale, out_dev, lse_dev, workspace_dev,
                  workspace_bytes, cuda_stream);
}
