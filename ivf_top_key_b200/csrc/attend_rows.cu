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
// and values; the products are mma.sync m16n8k16 (G <= 64 rows would leave a
// 128-row tcgen05 tile half empty or worse, and fp8 codes are widened in
// registers, between shared memory and the product).  Up to eight heads go to
// attend_few.cu: 4 x 131072 tokens of 8 key heads 317 us there, 356 us here.
//
// Measured: 8192 rows of 2048 of 131072 keys, one key head of 32 query heads:
// 1.30 ms, 8.6 GB of rows from L2 (6.6 TB/s) and 211 TFLOP/s.  It is the
// computing warps' latency that bounds it (two an SM quarter, what their
// registers leave): without the products the same copies take 1.06 ms.
//
// Work: tiles of keys (here 64, or 128 where that is at most 32 KB).  The CTAs
// (one per SM) divide all tiles of the batch evenly, whatever the lengths; a
// row whose tiles lie in several CTAs is joined by a second kernel from
// per-CTA partial results, always in tile order (no atomics on results: they
// do not depend on timing).  With several rows
// per CTA (prefill) whole rows are dealt out in turn, heads outermost, so
// that rows running at the same time read the same head's keys (L2), and
// only the last part wave is divided.
//
// In a CTA four warps copy, each a quarter of a tile's keys: one lane per key
// looks up where it lies (ids two batches of 32 keys ahead, the page one), then
// the warp copies the rows (cp.async, zeros for what is masked) into a ring of
// stages.  Eight warps compute: two groups of four take the row's tiles in
// turn, each warp its share of the tile's keys (or of the heads), with its own
// maximum, sum and output; they meet once per row.  Every warp follows the
// division of work by itself, a row at a time: what one warp does per tile
// bounds the tile rate (its instructions wait for one another, about 5 cycles
// each, and a look-up for memory).  (One warp that looked up all keys and told
// the others took 1500 cycles a tile; gathering rows by TMA, four an operation
// from one warp, 6500.)
#include <cmath>

#include "attend_rows.cuh"

namespace aiidx {
namespace {

constexpr int kWarps = 8;                       // that compute
constexpr int kCopiers = 4;                     // that look up and copy a quarter of a tile's keys each
constexpr int kThreads = (kWarps + kCopiers) * 32;
// ------------------------------------------------------------ shared memory
template <int D, bool FP8, int MT>
struct Layout {
  static constexpr int kRow = FP8 ? D : 2 * D;          // bytes of a key row
  static constexpr int kLine = kRow < 128 ? kRow : 128; // bytes of it that lie together
  static constexpr int kTile = kRow >= 256 ? 64 : 128;  // keys of a tile
  static constexpr int kKV = kTile * kRow;              // bytes of a K or V tile
  static constexpr int kQRow = 2 * D;
  static constexpr int kQ = 16 * MT * kQRow;
  static constexpr int kScales = FP8 ? 2 * kTile * 4 : 0;
  static constexpr int kWK = 4 / MT;                    // warps of a group along the keys
  static constexpr int kParts = 2 * kWK;                // states that meet per head row
  static constexpr int kState = D + 4;                  // floats: output, maximum, sum
  static constexpr int kMerge = kParts * 16 * MT * kState * 4;
  // 128 KB of keys and values, or what the rest leaves
  static constexpr int kRoom = (227 * 1024 - 768 - 2 * kQ - kMerge) / (2 * kKV + kScales + 32);
  static constexpr int kStages = kRoom < 131072 / (2 * kKV) ? kRoom : 131072 / (2 * kKV);
  static constexpr int kBars = 2 * kStages + 6;
  static constexpr int kBytes = kStages * (2 * kKV + kScales + 16) + 2 * kQ + kMerge + kBars * 8 + 16;
  static_assert(kBytes <= 227 * 1024 - 512, "shared memory");
  // 16-byte chunk c of tile row r: the eight rows of an ldmatrix fall on
  // different banks
  __device__ static uint32_t at(int r, int c) {
    if constexpr (kLine == 128) return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
  // 16-byte chunk c of query row r
  __device__ static uint32_t q_at(int r, int c) { return r * kQRow + ((c ^ (r & 7)) << 4); }
  // Tile row of column i of an 8-key product: for fp8 rows of 128 bytes such
  // that the rows of a quarter warp's 16-byte loads fall on different banks
  __device__ static constexpr int key(int i) {
    if constexpr (FP8 && kLine == 128) return ((i & 1) << 2) | (i >> 1);
    return i;
  }
};

template <int D, bool FP8, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend_rows(const RowsArgs a) {
  using L = Layout<D, FP8, MT>;
  constexpr int S = L::kStages;
  constexpr int WK = L::kWK;
  constexpr int kTile = L::kTile;
  constexpr int NK = kTile / WK;               // keys of a tile per computing warp
  constexpr int NB = NK < 32 ? NK : 32;        // of which at a time
  extern __shared__ __align__(128) uint8_t stages[];
  uint8_t* sq = stages + S * 2 * L::kKV;                        // [2] queries
  float* merge = reinterpret_cast<float*>(sq + 2 * L::kQ);
  float* scales = merge + L::kMerge / 4;                        // [S][2][64]
  uint32_t* reals = reinterpret_cast<uint32_t*>(scales + S * L::kScales / 4);  // [S][4] bit i of w: key 32 w + i is there
  uint64_t* full = reinterpret_cast<uint64_t*>(reals + S * 4);                                  // [S] tile landed
  uint64_t* empty = full + S;                                   // [S] tile read
  uint64_t* q_full = empty + S;                                 // [2] queries landed
  uint64_t* q_empty = q_full + 2;                               // [2] queries read
  uint64_t* joined = q_empty + 2;                               // [2] states written / read
  int* abort = reinterpret_cast<int*>(joined + 2);
  int* err = a.status;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_heads = a.n_heads;
  const int cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], kCopiers * 33);   // each lane's copies, each warp's bits
      mbar_init(&empty[i], kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], kCopiers * 32);
      mbar_init(&q_empty[i], kWarps);
    }
    mbar_init(&joined[0], kWarps);
    mbar_init(&joined[1], kWarps);
    *abort = 0;
    fence_mbar_init();
  }

  dependency_wait();
  Walk w;
  begin_walk<kThreads, D>(a, reinterpret_cast<int*>(merge) /* before the first row is joined */, err, &w);
  // the joining kernel may be set up now; it waits for this one to end
  dependency_launch();
  Share x;

  if (warp >= kWarps) {
    // ============================================================== copies
    // the computing warps take registers that copying does not need (8 x 216 +
    // 4 x 72 a lane, as many as the block was launched with: 12 x 168)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int cw = warp - kWarps;
    constexpr int kChunks = L::kRow / 16;            // 16-byte chunks of a key row
    constexpr int kStep = 32 / kChunks;              // rows that the warp copies at a time
    const int chunk = lane % kChunks, r_lane = lane / kChunks;
    const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * L::kRow;
    // what the joining kernel reads: the item that began before this CTA, or
    // -1 (0), whether it ends here (1), and the item that begins here and goes
    // on in the next CTA that has a share, or -1 (2)
    if (cw == 0 && lane == 0) *reinterpret_cast<int4*>(a.meta + cta * 4) = make_int4(-1, 1, -1, -1);
    __syncwarp();
    // A batch: 32 keys of this warp, that is one or two tiles of a share.
    constexpr int KW = kTile / kCopiers, BT = 32 / KW;
    const int sub = lane / KW, key = cw * KW + lane % KW;
    struct Batch {
      Share x;
      int t;          // first tile; x.t1 where there is none
      int seq, len;
      int tok;        // this lane's token, -1: none
    };
    bool more = w.next(a, &x);
    int seq = 0, len = 0, t_next = 0;
    auto enter = [&]() {
      seq = seq_of(a, x.row);
      len = len_of(a, x.row);
      t_next = x.t0;
    };
    if (more) enter();
    // step 1: the tokens of the next batch
    auto plan = [&](Batch& p) {
      p.tok = -1;
      p.len = 0;
      p.t = p.x.t1 = 0;
      if (!more) return;
      p.x = x;
      p.t = t_next;
      p.seq = seq;
      p.len = len;
      const int t = t_next + sub, at = t * kTile + key;
      if (t < x.t1) {
        if (!a.ids) p.tok = at < len ? at : -1;
        else if (at < a.n_ids) p.tok = a.ids[static_cast<int64_t>(x.row) * a.n_ids + at];
      }
      t_next += BT;
      if (t_next >= x.t1) {
        const int row = x.row;
        more = w.next(a, &x);
        t_next = x.t0;
        if (more && x.row != row) enter();
      }
    };
    // step 2: their pages
    auto page = [&](Batch& p) {
      if (p.tok >= p.len) {
        if (p.tok >= 0) atomicOr(err, AI_DEVFLAG_RANGE);
        p.tok = -1;
      }
      return p.tok >= 0 ? a.tables[static_cast<int64_t>(p.seq) * a.width + page_of(a, p.tok)] : -1;
    };
    Batch now, ahead;
    plan(now);
    int pg = page(now);
    plan(ahead);
    uint32_t n = 0, n_shares = 0;
    bool ok = true;
    int kv_head = 0;
    while (ok && now.t < now.x.t1) {
      const int next_pg = page(ahead);
      Batch later;
      plan(later);
      // step 3: their rows in the pool (-1: none), and the copies
      int row = -1;
      if (now.tok >= 0) {
        if (pg >= 0 && pg < a.n_pages) row = pg * a.page_size + (now.tok - page_of(a, now.tok) * a.page_size);
        else atomicOr(err, AI_DEVFLAG_RANGE);
      }
      const uint32_t real = __ballot_sync(0xffffffffu, row >= 0);
      if (now.t == now.x.t0) {
        kv_head = a.n_mb == 1 ? now.x.head : now.x.head / a.n_mb;
        if (cw == 0 && lane == 0 && now.x.slot >= 0) {
          const int item = now.x.row * n_heads + now.x.head;
          if (now.x.slot == 1) {
            a.meta[cta * 4 + 2] = item;
          } else {
            a.meta[cta * 4 + 0] = item;
            a.meta[cta * 4 + 1] = now.x.ends;
          }
        }
        const uint32_t qs = n_shares & 1;
        if (n_shares >= 2 && !__all_sync(0xffffffffu, mbar_wait(&q_empty[qs], (n_shares / 2 - 1) & 1, err, abort))) break;
        const int h0 = kv_head * a.G + (now.x.head - kv_head * a.n_mb) * a.mb_rows;
        const int n_rows = min(a.mb_rows, (kv_head + 1) * a.G - h0);
        const uint32_t dst = smem_u32(sq + qs * L::kQ);
        const uint16_t* src = a.q + (static_cast<int64_t>(now.x.row) * a.Hq + h0) * D;
        for (int i = cw * 32 + lane; i < 16 * MT * (D / 8); i += kCopiers * 32) {
          const int r = i / (D / 8), c = i % (D / 8);
          cp16z(dst + L::q_at(r, c), src + (r < n_rows ? r * D : 0) + c * 8, r < n_rows);
        }
        cp_async_mbar_arrive_noinc(&q_full[qs]);
        ++n_shares;
      }
      const uint8_t* kb = a.k + kv_head * L::kRow + chunk * 16;
      const uint8_t* vb = a.v + kv_head * L::kRow + chunk * 16;
#pragma unroll
      for (int j = 0; j < BT; ++j) {
        if (now.t + j >= now.x.t1) break;
        const uint32_t st = n % S;
        if (n >= S && !__all_sync(0xffffffffu, mbar_wait(&empty[st], (n / S - 1) & 1, err, abort))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if constexpr (KW == 32) reals[st * 4 + cw] = real;
          else reinterpret_cast<uint16_t*>(reals + st * 4)[cw] = static_cast<uint16_t>(real >> (j * 16));
        }
        // (a computing warp's keys may be several copying warps', and needs the
        // zeros of those that have none)
        if (NB > KW || (real >> (j * KW)) & (KW == 32 ? 0xffffffffu : 0xffffu)) {
          const uint32_t dst = smem_u32(stages + st * 2 * L::kKV);
#pragma unroll
          for (int i = 0; i < KW; i += kStep) {
            const int r = i + r_lane;
            const int src = __shfl_sync(0xffffffffu, row, j * KW + r);
            const int64_t off = src < 0 ? 0 : src * row_bytes;
            const uint32_t to = dst + L::at(cw * KW + r, chunk);
            cp16z(to, kb + off, src >= 0);
            cp16z(to + L::kKV, vb + off, src >= 0);
          }
          if constexpr (FP8) {
            const int64_t off = row < 0 ? 0 : static_cast<int64_t>(row) * a.Hkv + kv_head;
            const uint32_t to = smem_u32(scales + st * 2 * kTile + key);
            cp4z(to, a.ks + off, row >= 0);
            cp4z(to + kTile * 4, a.vs + off, row >= 0);
          }
        }
        cp_async_mbar_arrive_noinc(&full[st]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        ++n;
      }
      now = ahead;
      ahead = later;
      pg = next_pg;
    }
    cp_async_wait_all();
  } else {
    // ============================================================= compute
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int g = lane >> 2, t = lane & 3;
    const int group = warp >> 2, wm = warp % MT, wk = (warp & 3) / MT;
    const int part = group * WK + wk;              // which of the states of its head rows
    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m_run[2], l_run[2];
    float c2[2] = {a.c2, a.c2};                    // by row: scale * log2 e (fp8: and the queries' power of two)
    float base = -INFINITY, top = -INFINITY;       // fp8: see scale_base
    bool begun = false;
    // The maximum moves only when it grows by more than 2^kGrow: the weights
    // stay in range and most tiles leave o as it is.  fp8: weights are
    // 2^kLift e^(s - m) * (value scale / 2^base), in f16: 11 bits down to 2^-25
    // of the largest, smaller ones to within 2^-36 of it, and at most 2^15.
    constexpr float kGrow = FP8 ? 4.f : 8.f, kLift = 11.f;

    uint32_t n = 0, n_shares = 0;
    bool ok = true;
    while (ok && w.next(a, &x)) {
      const uint32_t qs = n_shares & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&q_full[qs], (n_shares / 2) & 1, err, abort))) break;
      {
        const uint8_t* q = sq + qs * L::kQ;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          if constexpr (!FP8) {
            ldsm4(qf[kk], smem_u32(q) + L::q_at(wm * 16 + (lane & 15), kk * 2 + (lane >> 4)));
          } else {
            // the product's sum over d in the order of the codes' 16-byte loads
            const int d = (kk / 4) * 64 + t * 16 + (kk % 4) * 4;
            const uint2 x = *reinterpret_cast<const uint2*>(q + L::q_at(wm * 16 + g, d / 8) + (d % 8) * 2);
            const uint2 y = *reinterpret_cast<const uint2*>(q + L::q_at(wm * 16 + g + 8, d / 8) + (d % 8) * 2);
            qf[kk][0] = x.x;
            qf[kk][1] = y.x;
            qf[kk][2] = x.y;
            qf[kk][3] = y.y;
          }
        }
        if constexpr (FP8) {
          // the codes are widened to f16, so the queries are f16 too: scaled by
          // a power of two that brings the row's largest to 2^14 .. 2^15 (exact;
          // what falls below f16's range is below 2^-39 of the largest)
          uint32_t mx[2] = {0, 0};
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = qf[kk][i] & 0x7fff7fffu;
              mx[i & 1] = max(mx[i & 1], max(x & 0xffffu, x >> 16));
            }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[i] = max(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = max(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            const int e = static_cast<int>(mx[i] >> 7);           // biased exponent
            const int up = e == 0 || e == 255 ? 0 : max(-100, min(100, 127 + 14 - e));
            const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            c2[i] = a.c2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
              for (int j = i; j < 4; j += 2)
                qf[kk][j] = pack_f16(__uint_as_float(qf[kk][j] << 16) * f, __uint_as_float(qf[kk][j] & 0xffff0000u) * f);
          }
          base = top = -INFINITY;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[qs]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m_run[0] = m_run[1] = -INFINITY;
        l_run[0] = l_run[1] = 0.f;
        begun = false;
      }
      // fp8, by block of a tile's keys: those of this log2 scale and more are done
      float far[NK / NB];
#pragma unroll
      for (int i = 0; i < NK / NB; ++i) far[i] = INFINITY;
      for (int tile = x.t0; tile < x.t1;) {
        const uint32_t st = n % S;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (n / S) & 1, err, abort))) {
          ok = false;
          break;
        }
        const uint8_t* stage = stages + st * 2 * L::kKV;
        const uint32_t sk = smem_u32(stage), sv = sk + L::kKV;
        bool again = false;
        if ((n & 1) == group) {
#pragma unroll
          for (int blk = 0; blk < NK / NB; ++blk) {
            const int k0 = wk * NK + blk * NB;      // first key of the block
            constexpr uint32_t kAll = NB == 32 ? 0xffffffffu : (1u << (NB % 32)) - 1;
            const uint32_t real = (reals[st * 4 + k0 / 32] >> (k0 % 32)) & kAll;  // its keys, one bit each
            if (real == 0 || (FP8 && far[blk] == -INFINITY)) continue;
            float left = -INFINITY;                 // fp8: keys below it need another pass
            float s[NB / 8][4];
#pragma unroll
            for (int j = 0; j < NB / 8; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
            if constexpr (!FP8) {
              // a step's keys are loaded while the products of the one before run
              uint32_t kf[2][NB / 16][4];
              auto load_k = [&](int kk) {
#pragma unroll
                for (int j = 0; j < NB / 16; ++j)
                  ldsm4(kf[kk & 1][j], sk + L::at(k0 + j * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)));
              };
              load_k(0);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                if (kk + 1 < D / 16) load_k(kk + 1);
#pragma unroll
                for (int j = 0; j < NB / 16; ++j) {
                  mma<false>(s[2 * j], qf[kk], kf[kk & 1][j][0], kf[kk & 1][j][1]);
                  mma<false>(s[2 * j + 1], qf[kk], kf[kk & 1][j][2], kf[kk & 1][j][3]);
                }
              }
            } else {
#pragma unroll
              for (int c4 = 0; c4 < D / 64; ++c4) {
#pragma unroll
                for (int j = 0; j < NB / 8; ++j) {
                  const uint4 x =
                      *reinterpret_cast<const uint4*>(stage + L::at(k0 + j * 8 + L::key(g), c4 * 4 + t));
                  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16x4(u[i], &b0, &b1);
                    mma<true>(s[j], qf[c4 * 4 + i], b0, b1);
                  }
                }
              }
            }
            // scale, mask and the running maximum
            const float* ksc = scales + st * 2 * kTile + k0;
            float mx[2] = {-INFINITY, -INFINITY};
            float lv[FP8 ? NB / 4 : 1], hi = -INFINITY, lo = INFINITY;   // fp8: log2 of the value scales
#pragma unroll
            for (int j = 0; j < NB / 8; ++j) {
              if constexpr (FP8) {
                const int i0 = j * 8 + L::key(2 * t), i1 = j * 8 + L::key(2 * t + 1);
                const float f0 = ksc[i0], f1 = ksc[i1];
                s[j][0] *= c2[0] * f0;
                s[j][1] *= c2[0] * f1;
                s[j][2] *= c2[1] * f0;
                s[j][3] *= c2[1] * f1;
                lv[2 * j] = __log2f(ksc[kTile + i0]);
                lv[2 * j + 1] = __log2f(ksc[kTile + i1]);
                hi = fmaxf(hi, fmaxf(lv[2 * j], lv[2 * j + 1]));
                lo = fminf(lo, fminf(lv[2 * j], lv[2 * j + 1]));
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) s[j][i] *= a.c2;
              }
            }
            if (real != kAll) {
#pragma unroll
              for (int j = 0; j < NB / 8; ++j) {
                const uint32_t bits = real >> (j * 8);
                const bool r0 = (bits >> L::key(2 * t)) & 1, r1 = (bits >> L::key(2 * t + 1)) & 1;
                s[j][0] = r0 ? s[j][0] : -INFINITY;
                s[j][1] = r1 ? s[j][1] : -INFINITY;
                s[j][2] = r0 ? s[j][2] : -INFINITY;
                s[j][3] = r1 ? s[j][3] : -INFINITY;
              }
            }
#pragma unroll
            for (int j = 0; j < NB / 8; ++j) {
              mx[0] = fmaxf(mx[0], fmaxf(s[j][0], s[j][1]));
              mx[1] = fmaxf(mx[1], fmaxf(s[j][2], s[j][3]));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
              mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            }
            const bool move0 = !begun ? mx[0] > -INFINITY : mx[0] > m_run[0] + kGrow || (m_run[0] == -INFINITY && mx[0] > -INFINITY);
            const bool move1 = !begun ? mx[1] > -INFINITY : mx[1] > m_run[1] + kGrow || (m_run[1] == -INFINITY && mx[1] > -INFINITY);
            float first = 1.f;                      // the sum takes a block's weights once
            if (FP8 && far[blk] != INFINITY) {
              first = 0.f;
              hi = lo = -INFINITY;
#pragma unroll
              for (int i = 0; i < NB / 4; ++i) {
                lv[i] = lv[i] < far[blk] ? lv[i] : -INFINITY;
                hi = fmaxf(hi, lv[i]);
              }
            }
            if (__any_sync(0xffffffffu, move0 || move1 || (FP8 && (hi > base || lo < base - kSpan)))) {
              const float m0 = move0 ? mx[0] : m_run[0], m1 = move1 ? mx[1] : m_run[1];
              const float f0 = move0 ? exp2_approx(m_run[0] - m0) : 1.f, f1 = move1 ? exp2_approx(m_run[1] - m1) : 1.f;
              m_run[0] = m0;
              m_run[1] = m1;
              float fe = 1.f;
              if constexpr (FP8) {
                float e = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
                e = ceilf(fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 2)));
                const float b = scale_base(e, base, far[blk] == INFINITY, &top);
                if (b != base) fe = pow2(base - b);
                base = b;
                const float low = scale_rest(e, b);
                bool more = false;
#pragma unroll
                for (int i = 0; i < NB / 4; ++i)
                  if (lv[i] < low) {
                    more |= lv[i] != -INFINITY;
                    lv[i] = -INFINITY;
                  }
                if (__any_sync(0xffffffffu, more)) {
                  left = low;
                  again = true;
                }
              }
              if (begun) {
                l_run[0] *= f0;
                l_run[1] *= f1;
                const float g0 = f0 * fe, g1 = f1 * fe;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                  o[i][0] *= g0;
                  o[i][1] *= g0;
                  o[i][2] *= g1;
                  o[i][3] *= g1;
                }
              }
            }
            begun = true;
            // a row without a finite score so far: exponents against 0 (all e^-inf = 0)
            const float mu[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0], m_run[1] == -INFINITY ? 0.f : m_run[1]};
            // the weights, rounded once (bf16; fp8: f16) for the product with v; their
            // sum is taken before that rounding.  (A second bf16 term, as for few heads,
            // would double the product where the computing warps are the bound.)
            uint32_t p[NB / 16][4];
            const float lift = kLift - (base == -INFINITY ? 0.f : base);
#pragma unroll
            for (int j = 0; j < NB / 8; ++j) {
              const float x0 = s[j][0] - mu[0], x1 = s[j][1] - mu[0], x2 = s[j][2] - mu[1], x3 = s[j][3] - mu[1];
              const float e0 = exp2_approx(x0), e1 = exp2_approx(x1), e2 = exp2_approx(x2), e3 = exp2_approx(x3);
              l_run[0] = FP8 ? fmaf(e0 + e1, first, l_run[0]) : l_run[0] + (e0 + e1);
              l_run[1] = FP8 ? fmaf(e2 + e3, first, l_run[1]) : l_run[1] + (e2 + e3);
              if constexpr (FP8) {
                const float v0 = lv[2 * j] + lift, v1 = lv[2 * j + 1] + lift;
                p[j / 2][(j & 1) * 2 + 0] = pack_f16(exp2_approx(x0 + v0), exp2_approx(x1 + v1));
                p[j / 2][(j & 1) * 2 + 1] = pack_f16(exp2_approx(x2 + v0), exp2_approx(x3 + v1));
              } else {
                p[j / 2][(j & 1) * 2 + 0] = pack_bf16(e0, e1);
                p[j / 2][(j & 1) * 2 + 1] = pack_bf16(e2, e3);
              }
            }
            // lane i gives the address of row i of an 8 x 8 block, in the keys' order
            const int vr = k0 + (lane & 8) + L::key(lane & 7);
            if constexpr (!FP8) {
              constexpr int kSteps = NB / 16 * (D / 16);
              uint32_t vf[3][4];
              auto load_v = [&](int u) {
                ldsm4t(vf[u % 3], sv + L::at(vr + u / (D / 16) * 16, u % (D / 16) * 2 + (lane >> 4)));
              };
              load_v(0);
              load_v(1);
#pragma unroll
              for (int u = 0; u < kSteps; ++u) {
                if (u + 2 < kSteps) load_v(u + 2);
                const int j = u / (D / 16), dd = u % (D / 16);
                mma<false>(o[2 * dd], p[j], vf[u % 3][0], vf[u % 3][1]);
                mma<false>(o[2 * dd + 1], p[j], vf[u % 3][2], vf[u % 3][3]);
              }
            } else {
              // 16-bit transposed loads bring two neighbouring codes of two keys;
              // accumulator 2 i holds the even, 2 i + 1 the odd d of 16-code chunk i
#pragma unroll
              for (int j = 0; j < NB / 16; ++j) {
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                  uint32_t b[4];
                  ldsm4t(b, sv + L::at(vr + j * 16, cc * 2 + (lane >> 4)));
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t even[2], odd[2];   // by key half
                    e4m3x4_to_f16x4(__byte_perm(b[2 * i], 0, 0x3120), &even[0], &odd[0]);
                    e4m3x4_to_f16x4(__byte_perm(b[2 * i + 1], 0, 0x3120), &even[1], &odd[1]);
                    mma<true>(o[(cc * 2 + i) * 2], p[j], even[0], even[1]);
                    mma<true>(o[(cc * 2 + i) * 2 + 1], p[j], odd[0], odd[1]);
                  }
                }
              }
            }
            far[blk] = left;
          }
        }
        if (FP8 && again) continue;
#pragma unroll
        for (int i = 0; i < NK / NB; ++i) far[i] = INFINITY;
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        ++tile;
        ++n;
      }
      if (!ok) break;
      {
        // the row sums over the four lanes of a row, then over the states
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 1);
          l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], 2);
        }
        if constexpr (FP8) {
          const float f = base == -INFINITY ? 0.f : exp2_approx(base - kLift);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= f;
            o[i][1] *= f;
            o[i][2] *= f;
            o[i][3] *= f;
          }
        }
        // the states of the row before have been read
        if (n_shares > 0 && !__all_sync(0xffffffffu, mbar_wait(&joined[1], (n_shares - 1) & 1, err, abort))) break;
        float* mine = merge + (part * MT + wm) * 16 * L::kState;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float* to = mine + (g + half * 8) * L::kState;
          if constexpr (!FP8) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(to + i * 8 + 2 * t) = make_float2(o[i][2 * half], o[i][2 * half + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              *reinterpret_cast<float4*>(to + i * 16 + 4 * t) =
                  make_float4(o[2 * i][2 * half], o[2 * i + 1][2 * half], o[2 * i][2 * half + 1], o[2 * i + 1][2 * half + 1]);
          }
          if (t == 0) *reinterpret_cast<float2*>(to + D) = make_float2(m_run[half], l_run[half]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[0]);
        if (!__all_sync(0xffffffffu, mbar_wait(&joined[0], n_shares & 1, err, abort))) break;
        // each thread joins a piece of one head row
        constexpr int kPer = 16 * MT * D / (kWarps * 32);   // its columns: 8 to 32 (D = 64: 4 to 16)
        const int r = tid * kPer / D, c0 = tid * kPer % D;
        const float* from = merge + ((r >> 4) * 16 + (r & 15)) * L::kState;
        constexpr int kNext = MT * 16 * L::kState;          // the next part's state of the row
        float wgt[L::kParts], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < L::kParts; ++i) m = fmaxf(m, from[i * kNext + D]);
        const float mz = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < L::kParts; ++i) {
          wgt[i] = exp2_approx(from[i * kNext + D] - mz);
          l += from[i * kNext + D + 1] * wgt[i];
        }
        const int kv_head = a.n_mb == 1 ? x.head : x.head / a.n_mb;
        const int h0 = kv_head * a.G + (x.head - kv_head * a.n_mb) * a.mb_rows;
        const bool used = r < min(a.mb_rows, (kv_head + 1) * a.G - h0);
        const float inv = x.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
#pragma unroll
        for (int c = 0; c < kPer; c += 4) {
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < L::kParts; ++i) {
            const float4 z = *reinterpret_cast<const float4*>(from + i * kNext + c0 + c);
            y.x = fmaf(z.x, wgt[i], y.x);
            y.y = fmaf(z.y, wgt[i], y.y);
            y.z = fmaf(z.z, wgt[i], y.z);
            y.w = fmaf(z.w, wgt[i], y.w);
          }
          // a head that saw nothing, or whose scores are all -inf, is zero whatever the values hold
          if (x.slot < 0 && l == 0.f) y = make_float4(0.f, 0.f, 0.f, 0.f);
          if (used) {
            if (x.slot < 0)
              *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(x.row) * a.Hq + h0 + r) * D + c0 + c) =
                  make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
            else
              *reinterpret_cast<float4*>(a.part + (static_cast<int64_t>(cta * 2 + x.slot) * 16 * MT + r) * L::kState +
                                         c0 + c) = y;
          }
        }
        if (used && c0 == 0) {
          if (x.slot >= 0)
            *reinterpret_cast<float2*>(a.part + (static_cast<int64_t>(cta * 2 + x.slot) * 16 * MT + r) * L::kState + D) =
                make_float2(m, l);
          else if (a.lse)
            a.lse[static_cast<int64_t>(x.row) * a.Hq + h0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&joined[1]);
      }
      ++n_shares;
    }
  }
}

// Head rows of a partial result, padded to the kernels' tiles.
int rows_per_slot(int mb_rows) { return mb_rows <= kFewHeads ? 8 : (mb_rows <= 16 ? 16 : (mb_rows <= 32 ? 32 : 64)); }

// Joins the parts of a row that begins in CTA blockIdx.x and goes on in the
// following ones; blockIdx.y is the row within the block of query heads.  A
// thread takes a part's maximum and sum, then a column: what is read in turn
// is read by many at once (one part after another took 0.4 us each).
// Launched to start while the partial kernel ends (programmatic dependence):
// it waits for it before it reads.
constexpr int kJoin = 128;
template <int D>
__global__ void __launch_bounds__(kJoin) k_join_rows(const RowsArgs a, int n_ctas, int slot_rows) {
  __shared__ float sh_w[kJoin], sh_red[kJoin / 32], sh_o[kJoin];
  __shared__ int sh_end;
  dependency_wait();
  const int c = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
  const int item = a.meta[c * 4 + 2];
  if (item < 0) return;
  const int n_heads = a.Hkv * a.n_mb;
  const int head = item % n_heads, row = item / n_heads;
  const int h = head / a.n_mb;
  const int h0 = h * a.G + (head % a.n_mb) * a.mb_rows;
  if (r >= min(a.mb_rows, (h + 1) * a.G - h0)) return;
  auto part = [&](int n) {   // of CTA n; the row's first part is its CTA's second slot
    return a.part + (static_cast<int64_t>(n * 2 + (n == c)) * slot_rows + r) * (D + 4);
  };
  constexpr int kCols = kJoin / D;     // threads per column: parts n0 + tid / D, + kCols, ..
  const int d = tid % D, sub = tid / D;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int n0 = c, end = n_ctas; n0 < end; n0 += kJoin) {
    // up to kJoin parts: CTAs n0 .. ; the row ends in the first that says so
    const int n = n0 + tid;
    float pm = -INFINITY, pl = 0.f;
    if (tid == 0) sh_end = n_ctas;
    __syncthreads();
    if (n < n_ctas) {
      const int2 x = *reinterpret_cast<const int2*>(a.meta + n * 4);
      if (n == c || x.x == item) {     // (a CTA without a share has none)
        const float2 ml = *reinterpret_cast<const float2*>(part(n) + D);
        pm = ml.x;
        pl = ml.y;
        if (n > c && x.y) atomicMin(&sh_end, n + 1);
      }
    }
    __syncthreads();
    end = min(end, sh_end);
    if (n >= end) {
      pm = -INFINITY;
      pl = 0.f;
    }
    // the new maximum, the parts' weights and their sum
    float mx = pm;
    for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    if ((tid & 31) == 0) sh_red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(fmaxf(fmaxf(sh_red[0], sh_red[1]), fmaxf(sh_red[2], sh_red[3])), m);
    const float mz = mn == -INFINITY ? 0.f : mn;
    const float w = exp2_approx(pm - mz);
    sh_w[tid] = pl == 0.f ? -1.f : w;  // -1: nothing seen, its output may not be written
    float sum = pl == 0.f ? 0.f : pl * w;
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    __syncthreads();
    if ((tid & 31) == 0) sh_red[tid >> 5] = sum;
    __syncthreads();
    const float f = exp2_approx(m - mz);
    l = l * f + ((sh_red[0] + sh_red[1]) + (sh_red[2] + sh_red[3]));
    o *= f;
    m = mn;
    const int count = min(end - n0, kJoin);
#pragma unroll 8
    for (int i = sub; i < count; i += kCols) {
      const float wi = sh_w[i];
      if (!(wi < 0.f)) o = fmaf(part(n0 + i)[d], wi, o);
    }
    __syncthreads();
  }
  if constexpr (kCols > 1) {
    sh_o[tid] = o;
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int i = 1; i < kCols; ++i) o += sh_o[i * D + d];
  }
  const __nv_bfloat16 b = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
  a.out[(static_cast<int64_t>(row) * a.Hq + h0 + r) * D + d] = *reinterpret_cast<const uint16_t*>(&b);
  if (a.lse && d == 0)
    a.lse[static_cast<int64_t>(row) * a.Hq + h0 + r] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D, bool FP8, int MT>
cudaError_t launch_mt(const RowsArgs& a, int grid, cudaStream_t st) {
  using L = Layout<D, FP8, MT>;
  static ReadyOnce ready;
  const cudaError_t e = ready.shared_memory(k_attend_rows<D, FP8, MT>, L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(k_attend_rows<D, FP8, MT>, dim3(grid), dim3(kThreads), L::kBytes, st, a);
}

template <int D, bool FP8>
cudaError_t launch_d(const RowsArgs& a, int grid, cudaStream_t st) {
  cudaError_t e;
  if (a.mb_rows <= kFewHeads) e = launch_rows_few(a, D, FP8, grid, st);
  else if (a.mb_rows <= 16) e = launch_mt<D, FP8, 1>(a, grid, st);
  else if (a.mb_rows <= 32) e = launch_mt<D, FP8, 2>(a, grid, st);
  else e = launch_mt<D, FP8, 4>(a, grid, st);
  if (e != cudaSuccess) return e;
  return launch_after(k_join_rows<D>, dim3(grid, a.mb_rows), dim3(kJoin), 0, st, a, grid, rows_per_slot(a.mb_rows));
}

int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

// The largest grid (partial results are sized for it).
int max_grid() { return device_sms(); }

int64_t workspace_for(int Hq, int Hkv, int D) {
  const int G = Hq / Hkv;
  const int mb = (G + 63) / 64;
  const int64_t g = max_grid();
  return g * 16 + g * 2 * rows_per_slot((G + mb - 1) / mb) * (D + 4) * 4;
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
  if (static_cast<int64_t>(R) * c->n_kv_heads * n_mb > 0x3fffffff) return fail(AI_ERR_ARG, "too many rows times key heads");
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
  a.n_heads = a.Hkv * n_mb;
  a.n_seqs = c->n_seqs;
  a.width = c->max_pages;
  a.n_pages = c->n_pages;
  a.page_size = c->page_size;
  int s = 0;
  while ((int64_t(1) << s) < c->page_size) ++s;
  a.page_shift = 31 + s;
  a.page_mul = ((uint64_t(1) << a.page_shift) + c->page_size - 1) / c->page_size;
  a.tile = a.mb_rows <= kFewHeads ? rows_few_tile() : (c->head_dim * es >= 256 ? 64 : 128);  // Layout::kTile
  // measured: about 1.5 us an item; 0.2 us a tile of 32 keys, 0.4 to 0.7 us a
  // larger one
  a.over = a.mb_rows <= kFewHeads ? 7 : 3;
  a.nt_ids = static_cast<int>((static_cast<int64_t>(n_ids) + a.tile - 1) / a.tile);
  a.c2 = scale * kLog2e;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = c->status ? c->status : default_status();
  if (!a.status) return fail(AI_ERR_CUDA, "the device's status word was not found");
  const int64_t most = ids ? n_ids : static_cast<int64_t>(c->max_pages) * c->page_size;
  const int64_t tiles = static_cast<int64_t>(R) * a.Hkv * n_mb * ((most + a.tile - 1) / a.tile);
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
  if (T > 0 && !ids_dev) return fail(AI_ERR_ARG, "null pointer argument");
  if (k <= 0) return fail(AI_ERR_ARG, "k must be positive");
  return run_rows(cache, layer, q_dev, T, n_heads, ids_dev, k, seqs_dev, scale, out_dev, lse_dev, workspace_dev,
                  workspace_bytes, cuda_stream);
}
