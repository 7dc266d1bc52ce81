// Shared by the kernels that attend for single rows over a paged cache: their
// arguments, warp-level products, the division of work among CTAs.
#pragma once

#include "../../include/ai_index.h"
#include "common.cuh"
#include "kernels.h"

namespace aiidx {

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
  int R, n_ids, nt_ids, Hq, Hkv, G;
  int n_mb, mb_rows;        // row blocks per key head, query heads per block
  int n_heads;              // Hkv * n_mb
  int n_seqs, width, n_pages, page_size;
  int tile;                 // keys of a tile
  int over;                 // what an item costs besides its tiles, in tiles
  uint64_t page_mul;        // token / page_size = token * page_mul >> page_shift
  int page_shift;
  float c2;                 // scale * log2 e
  uint16_t* out;            // [R, Hq, D] bf16
  float* lse;               // [R, Hq] or nullptr
  float* part;              // partial results: [2 * grid][16 MT][D + 4]
  int32_t* meta;            // [grid][4]
  int32_t* status;
};

namespace {

// ------------------------------------------------------------- warp products
template <bool F16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
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
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Four e4m3 codes (low byte first) to two pairs of f16 values, exactly.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t* lo, uint32_t* hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(*lo), "=r"(*hi)
      : "r"(codes));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 or 4 bytes to shared memory, zeros where !real.
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4z(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

// fp8: weights times value scales are f16 for the product with v, held against
// 2^base, which follows the tiles' largest value scales: up at once, down where a
// tile's is 2^kFall lower, so that a few keys of far larger scales (or zeros, whose
// scale is 1) do not take the others' bits.  Keys whose scales are more than
// 2^kSpan below it have a pass of their own over the tile.  The output so far,
// fp32, is rescaled with base, exactly, and stays in range: base keeps within 60
// of its largest (top).  e: log2 of the largest scale of a tile, rounded up.
constexpr float kFall = 6.f, kSpan = 10.f;
__device__ __forceinline__ float scale_base(float e, float base, bool first_pass, float* top) {
  *top = fmaxf(*top, e);
  if (e > base) return e;
  return e != -INFINITY && (!first_pass || e < base - kFall) ? fmaxf(e, *top - 60.f) : base;
}
// The log2 scale below which a tile's keys are left for another pass.  Every pass
// takes the largest left, so there are at most as many as keys; finite, also
// where a scale is infinite, as infinity stands for a first pass.
__device__ __forceinline__ float scale_rest(float e, float base) { return fminf(fminf(base - kSpan, e - 1.f), 1e30f); }
// 2^x for a whole x up to 127; 0 below -126
__device__ __forceinline__ float pow2(float x) { return __int_as_float(max(0, static_cast<int>(x) + 127) << 23); }

// ----------------------------------------------------------- division of work
// Division of a token (< 2^31) by the page size: with s = ceil(log2 d),
// m = ceil(2^(31 + s) / d) < 2^32 the quotient is exactly n m >> (31 + s)
// (Granlund and Montgomery, 1994).
__device__ __forceinline__ int page_of(const RowsArgs& a, int tok) {
  return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(tok)) * a.page_mul >> a.page_shift);
}
__device__ __forceinline__ int seq_of(const RowsArgs& a, int row) {
  return a.seqs ? a.seqs[row] : row * a.seq_mul;
}
__device__ __forceinline__ int len_of(const RowsArgs& a, int row) {
  const int s = seq_of(a, row);
  if (s < 0 || s >= a.n_seqs) return 0;
  const int64_t most = static_cast<int64_t>(a.width) * a.page_size;
  const int n = a.lens[s];
  if (n < 0 || n > most) atomicOr(a.status, AI_DEVFLAG_RANGE);
  return n < 0 ? 0 : (n > most ? static_cast<int>(most) : n);
}
__device__ __forceinline__ int tiles_of(const RowsArgs& a, int row) {
  return static_cast<int>((static_cast<uint32_t>(len_of(a, row)) + a.tile - 1) / a.tile);  // (past 2^31)
}

// A share of one item: tiles [t0, t1) of a row and a (key head, row block).
struct Share {
  int row, head, t0, t1;
  int slot;     // -1: the whole item; 0 / 1: partial result slot
  bool ends;    // the item's last tile is in it
};

// The shares of a CTA in order: whole items dealt out in turn (item it, it +
// grid, .. < n_whole; heads outermost), then the tiles [b, b1) of the divided
// items, which follow one another.  Every warp runs its own.
struct Walk {
  int it, n_whole;
  int64_t left;        // tiles of the divided items that are still to come
  int row, head;       // of the next divided item
  int tile, n_tiles;   // its next tile, and its tiles

  __device__ bool next(const RowsArgs& a, Share* s) {
    if (it < n_whole) {
      s->head = it / a.R;
      s->row = it - s->head * a.R;
      s->t0 = 0;
      s->t1 = a.nt_ids;
      s->slot = -1;
      s->ends = true;
      it += gridDim.x;
      return true;
    }
    if (left <= 0) return false;
    s->row = row;
    s->head = head;
    s->t0 = tile;
    s->ends = left >= n_tiles - tile;
    s->t1 = s->ends ? n_tiles : tile + static_cast<int>(left);
    // begun in an earlier CTA: its first slot; goes on in a later one: its second
    s->slot = tile > 0 ? 0 : (s->ends ? -1 : 1);
    left -= s->t1 - tile;
    tile = 0;
    if (a.ids) {       // heads outermost
      if (++row == a.R) {
        row = 0;
        ++head;
      }
    } else if (++head == a.n_heads) {
      head = 0;
      if (left > 0) {
        do ++row;
        while (row < a.R && tiles_of(a, row) == 0);
        n_tiles = row < a.R ? tiles_of(a, row) : 1;
      }
    }
    return true;
  }
};

// Block-wide sum and exclusive prefix of one int64 per thread.
template <int kThreads>
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

// This CTA's walk, by all its threads; rows that see nothing are written on
// the way.  sh_none: kThreads ints of shared memory.
template <int kThreads, int D>
__device__ void begin_walk(const RowsArgs& a, int* sh_none, int* err, Walk* out) {
  __shared__ int64_t sh_scan[kThreads / 32];
  __shared__ int64_t sh_part[2];   // this CTA's tiles of the divided items: first, end
  __shared__ Walk sh_w;
  __shared__ int sh_n_none;
  const int tid = threadIdx.x, grid = gridDim.x, cta = blockIdx.x;
  const int n_heads = a.n_heads;
  auto nothing = [&](int row, int first, int step) {   // zeros, and the log of an empty sum
    const int64_t at = static_cast<int64_t>(row) * a.Hq;
    for (int j = first; j < a.Hq * D / 8; j += step)
      reinterpret_cast<uint4*>(a.out + at * D)[j] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int j = first; j < a.Hq; j += step) a.lse[at + j] = -INFINITY;
    const int s = seq_of(a, row);
    if (first == 0 && (s < 0 || s >= a.n_seqs)) atomicOr(err, AI_DEVFLAG_RANGE);
  };
  if (tid == 0) {
    sh_w.it = cta;
    sh_w.n_whole = 0;
    sh_n_none = 0;
  }
  if (a.ids) {
    if (tid == 0) {
      const int64_t items = static_cast<int64_t>(a.R) * n_heads;
      const int n_whole = static_cast<int>(items / grid) * grid;
      const int64_t total = (items - n_whole) * a.nt_ids;
      const int64_t first = total * cta / grid, item = n_whole + first / a.nt_ids;
      sh_part[0] = first;
      sh_part[1] = total * (cta + 1) / grid;
      sh_w.n_whole = n_whole;
      sh_w.head = static_cast<int>(item / a.R);
      sh_w.row = static_cast<int>(item % a.R);
      sh_w.tile = static_cast<int>(first % a.nt_ids);
      sh_w.n_tiles = a.nt_ids;
    }
    __syncthreads();
  } else {
    // An item costs its tiles and, once, about a.over more (queries, states,
    // results): the CTAs divide that sum evenly, and a CTA's tiles are those
    // whose cost lies in its part.  `mine` tiles of row r behind t0 tiles and c0
    // cost of all heads: where the part's ends lie in the row.
    auto locate = [&](int r, int64_t mine, int64_t t0, int64_t c0, int64_t cost) {
      const int64_t n = mine + a.over;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t at = cost * (cta + u) / grid - c0;
        if (mine == 0 || at < 0 || at >= n * n_heads) continue;
        const int64_t head = at / n, rest = at - head * n - a.over;
        const int tile = rest > 0 ? static_cast<int>(rest) : 0;
        sh_part[u] = t0 + head * mine + tile;
        if (u == 0) {
          sh_w.row = r;
          sh_w.head = static_cast<int>(head);
          sh_w.tile = tile;
          sh_w.n_tiles = static_cast<int>(mine);
        }
      }
    };
    if (a.R <= 32) {
      if (tid < 32) {   // by one warp, without the block's barriers
        const int64_t mine = tid < a.R ? tiles_of(a, tid) : 0;
        const uint32_t some = __ballot_sync(0xffffffffu, mine > 0);
        int64_t inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (tid >= o) inc += y;
        }
        const int64_t total = __shfl_sync(0xffffffffu, inc, 31);
        const int64_t cost = (total + static_cast<int64_t>(__popc(some)) * a.over) * n_heads;
        if (tid < 2) sh_part[tid] = total * n_heads;   // a part that begins or ends behind the last tile
        __syncwarp();
        const int64_t t0 = (inc - mine) * n_heads;
        locate(tid, mine, t0, t0 + static_cast<int64_t>(__popc(some & ((1u << tid) - 1))) * a.over * n_heads, cost);
        for (uint32_t none = __ballot_sync(0xffffffffu, tid < a.R && mine == 0 && tid % grid == cta); none;
             none &= none - 1)
          nothing(__ffs(none) - 1, tid, 32);
      }
      __syncthreads();
    } else {
      // the sums, then the rows (a second pass over the lengths)
      int64_t total = 0, n_rows = 0;
      for (int r0 = 0; r0 < a.R; r0 += kThreads) {
        int64_t tiles, rows;
        const int64_t x = r0 + tid < a.R ? tiles_of(a, r0 + tid) : 0;
        block_scan<kThreads>(x, &tiles, sh_scan);
        block_scan<kThreads>(x > 0, &rows, sh_scan);
        total += tiles;
        n_rows += rows;
      }
      const int64_t cost = (total + n_rows * a.over) * n_heads;
      if (tid < 2) sh_part[tid] = total * n_heads;
      __syncthreads();
      int64_t tiles_seen = 0, rows_seen = 0;
      for (int r0 = 0; r0 < a.R; r0 += kThreads) {
        const int r = r0 + tid;
        int64_t tiles, rows;
        const int64_t mine = r < a.R ? tiles_of(a, r) : 0;
        const int64_t t0 = (tiles_seen + block_scan<kThreads>(mine, &tiles, sh_scan)) * n_heads;
        const int64_t before = rows_seen + block_scan<kThreads>(mine > 0, &rows, sh_scan);
        locate(r, mine, t0, t0 + before * a.over * n_heads, cost);
        tiles_seen += tiles;
        rows_seen += rows;
        if (r < a.R && mine == 0 && r % grid == cta) sh_none[atomicAdd(&sh_n_none, 1)] = r;
        __syncthreads();
        for (int i = 0; i < sh_n_none; ++i) nothing(sh_none[i], tid, kThreads);
        __syncthreads();
        if (tid == 0) sh_n_none = 0;
      }
      __syncthreads();
    }
  }
  *out = sh_w;
  out->left = sh_part[1] - sh_part[0];
}

}  // namespace

// Query heads per key head up to which launch_rows_few takes a call.
constexpr int kFewHeads = 8;
// The partial kernel of a call with a.mb_rows <= kFewHeads, on `grid` CTAs;
// partial results have 8 rows a slot.
cudaError_t launch_rows_few(const RowsArgs& a, int D, bool fp8, int grid, cudaStream_t st);
int rows_few_tile();  // keys of its tiles

}  // namespace aiidx
