// Attention of single rows over a paged cache where at most eight query heads
// share a key head (see attend_rows.cu for the formulas and the division of
// work).
//
// With so few heads the keys are the rows of the products and the heads their
// eight columns:  S^T = K Q^T  (16 keys x 8 heads),  O^T += V^T P^T  (16 values
// of d x 8 heads): half the products, accumulators and registers of heads as
// 16 rows.  K comes from shared memory by ldmatrix, V by transposed ldmatrix,
// P^T from the score accumulators through movmatrix.  fp8 codes are widened to
// f16 on the way (one conversion of two codes each).
//
// A tile is 32 keys and one warp's work from its look-up to its weights: each
// of kCopiers copying warps takes every kCopiers-th tile (lane = key: id, page,
// row), each computing warp every kComp-th.
// Computing warps take the queries from memory themselves, one row ahead, and
// hand over their states in two buffers that joining warps read, so that
// no row waits for the one before it.
//
// Measured: 4 x 131072 tokens of 8 key heads, bf16: 320 us, 6.7 TB/s (a plain
// read of the same bytes); 48 sequences of up to 8192 tokens, fp8: 98 to 102 us,
// 4.5 TB/s.  What bounds fp8 is the widening: half of the issue slots and 46 % of
// the ALU slots (tiles of 64 keys and ten computing warps measured the same).
#include "attend_rows.cuh"

namespace aiidx {
namespace {

constexpr int kTile = 32;

template <int D, bool FP8>
struct Few {
  static constexpr int kRow = FP8 ? D : 2 * D;          // bytes of a key row
  static constexpr int kLine = kRow < 128 ? kRow : 128; // bytes of it that lie together
  static constexpr int kKV = kTile * kRow;
  // sixteen warps at most: 128 registers each
  static constexpr int kComp = kRow > 64 ? 8 : 10;
  static constexpr int kCopiers = kRow > 64 ? 4 : 5;
  static constexpr int kJoiners = kRow > 64 ? 2 : 1;
  static constexpr int kThreads = (kComp + kCopiers + kJoiners) * 32;
  // a multiple of both, so that a stage is always the same two warps': each
  // waits for every phase of its barriers in turn
  static constexpr int kStages = kRow > 128 ? 8 : (kRow > 64 ? 16 : 20);
  static_assert(kStages % kComp == 0 && kStages % kCopiers == 0, "stages");
  static constexpr int kScales = FP8 ? 2 * kTile * 4 : 0;
  static constexpr int kState = D + 4;                  // floats: output, maximum, sum
  static constexpr int kStates = kComp * 8 * kState;    // of a row
  static constexpr int kBars = 2 * kStages + 4;
  static constexpr int kBytes = kStages * (2 * kKV + kScales + 4) + 2 * kStates * 4 + kBars * 8 + 16;
  static_assert(kBytes <= 227 * 1024 - 512, "shared memory");
  // 16-byte chunk c of tile row r: the eight rows of an ldmatrix fall on
  // different banks
  __device__ static uint32_t at(int r, int c) {
    if constexpr (kLine == 128) return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  }
  // Tile row of row i of an 8-key block: for fp8 rows of 128 bytes such that
  // the rows of a quarter warp's 16-byte loads fall on different banks
  __device__ static constexpr int key(int i) {
    if constexpr (FP8 && kLine == 128) return ((i & 1) << 2) | (i >> 1);
    return i;
  }
};

// 8 x 8 block of 16-bit values, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Few<D, FP8>::kThreads, 1) k_attend_few(const RowsArgs a) {
  using L = Few<D, FP8>;
  constexpr int S = L::kStages;
  constexpr int kComp = L::kComp, kCopiers = L::kCopiers, kJoiners = L::kJoiners;
  extern __shared__ __align__(128) uint8_t stages[];
  float* states = reinterpret_cast<float*>(stages + S * 2 * L::kKV);           // [2][kComp][8][D + 4]
  float* scales = states + 2 * L::kStates;                                     // [S][2][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + S * L::kScales / 4);   // [S] tile landed
  uint64_t* empty = full + S;                                                  // [S] tile read
  uint64_t* st_full = empty + S;                                               // [2] states written
  uint64_t* st_free = st_full + 2;                                             // [2] states read
  uint32_t* reals = reinterpret_cast<uint32_t*>(st_free + 2);                  // [S] bit i: key i of the tile is there
  int* abort = reinterpret_cast<int*>(reals + S);
  int* err = a.status;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 33);   // each lane's copies, and the bits
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&st_full[i], kComp);
      mbar_init(&st_free[i], kJoiners);
    }
    *abort = 0;
    fence_mbar_init();
  }
  dependency_wait();
  Walk w;
  begin_walk<L::kThreads, D>(a, reinterpret_cast<int*>(states) /* before the first state */, err, &w);
  // the joining kernel may be set up now; it waits for this one to end
  dependency_launch();
  Share x;
  // an item of one tile is finished by the warp that computes it
  auto single = [](const Share& s) { return s.slot < 0 && s.t1 - s.t0 == 1; };

  if (warp >= kComp + kCopiers) {
    // ============================================================= joining
    const int j = tid - (kComp + kCopiers) * 32;
    const int c0 = (j % 8) * 4;                     // columns c0 + 32 i
    uint32_t share = 0;
    while (w.next(a, &x)) {
      if (single(x)) continue;
      const uint32_t buf = share & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&st_full[buf], (share >> 1) & 1, err, abort))) break;
      constexpr int kNext = 8 * L::kState;
#pragma unroll
      for (int r = j / 8; r < 8; r += kJoiners * 4) {
        const float* from = states + buf * L::kStates + r * L::kState;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < kComp; ++i) m = fmaxf(m, from[i * kNext + D]);
        const float mz = m == -INFINITY ? 0.f : m;
        float4 y[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) y[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kComp; ++i) {
          const float2 ml = *reinterpret_cast<const float2*>(from + i * kNext + D);
          if (ml.y == 0.f) continue;                  // nothing seen: its output is not written
          const float f = exp2_approx(ml.x - mz);
          l += ml.y * f;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const float4 z = *reinterpret_cast<const float4*>(from + i * kNext + c * 32 + c0);
            y[c].x = fmaf(z.x, f, y[c].x);
            y[c].y = fmaf(z.y, f, y[c].y);
            y[c].z = fmaf(z.z, f, y[c].z);
            y[c].w = fmaf(z.w, f, y[c].w);
          }
        }
        if (r < a.G) {
          const int64_t at = static_cast<int64_t>(x.row) * a.Hq + x.head * a.G + r;
          if (x.slot < 0) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
              *reinterpret_cast<uint2*>(a.out + at * D + c * 32 + c0) =
                  make_uint2(pack_bf16(y[c].x * inv, y[c].y * inv), pack_bf16(y[c].z * inv, y[c].w * inv));
            if (a.lse && c0 == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else {
            float* part = a.part + (static_cast<int64_t>(cta * 2 + x.slot) * 8 + r) * L::kState;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) *reinterpret_cast<float4*>(part + c * 32 + c0) = y[c];
            if (c0 == 0) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&st_free[buf]);
      ++share;
    }
  } else if (warp >= kComp) {
    // ============================================================== copies
    const int cw = warp - kComp;
    constexpr int kChunks = L::kRow / 16;            // 16-byte chunks of a key row
    constexpr int kStep = 32 / kChunks;              // rows that the warp copies at a time
    const int chunk = lane % kChunks, r_lane = lane / kChunks;
    const int64_t row_bytes = static_cast<int64_t>(a.Hkv) * L::kRow;
    // what the joining kernel reads: the item that began before this CTA, or
    // -1 (0), whether it ends here (1), and the item that begins here and goes
    // on in the next CTA that has a share, or -1 (2)
    if (cw == 0 && lane == 0) *reinterpret_cast<int4*>(a.meta + cta * 4) = make_int4(-1, 1, -1, -1);
    __syncwarp();
    bool more = true;
    int seq = 0, len = 0, t = 0, at_row = -1;
    uint32_t n0 = 0;                                 // number of the share's first tile in this CTA
    auto enter = [&]() {                             // the next share that has a tile of this warp's
      do {
        more = w.next(a, &x);
        if (!more) return;
        if (cw == 0 && lane == 0 && x.slot >= 0) {
          const int item = x.row * a.Hkv + x.head;
          if (x.slot == 1) {
            a.meta[cta * 4 + 2] = item;
          } else {
            a.meta[cta * 4 + 0] = item;
            a.meta[cta * 4 + 1] = x.ends;
          }
        }
        t = x.t0 + static_cast<int>((cw + kCopiers - n0 % kCopiers) % kCopiers);
        n0 += x.t1 - x.t0;
      } while (t >= x.t1);
      if (x.row != at_row) {
        seq = seq_of(a, x.row);
        len = len_of(a, x.row);
        at_row = x.row;
      }
    };
    enter();
    struct Batch {
      uint32_t n;      // number of the tile
      int head, seq, len;
      int tok;         // this lane's token, -1: none
      bool there;
    };
    // step 1: the tokens of this warp's next tile
    auto plan = [&](Batch& p) {
      p.there = more;
      p.tok = -1;
      p.len = 0;
      if (!more) return;
      p.n = n0 - (x.t1 - t);
      p.head = x.head;
      p.seq = seq;
      p.len = len;
      const int at = t * kTile + lane;
      if (!a.ids) p.tok = at < len ? at : -1;
      else if (at < a.n_ids) p.tok = a.ids[static_cast<int64_t>(x.row) * a.n_ids + at];
      t += kCopiers;
      if (t >= x.t1) enter();
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
    while (now.there) {
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
      const uint32_t st = now.n % S;
      if (now.n >= S && !__all_sync(0xffffffffu, mbar_wait(&empty[st], (now.n / S - 1) & 1, err, abort))) break;
      if (lane == 0) reals[st] = real;
      if (real) {
        const uint32_t dst = smem_u32(stages + st * 2 * L::kKV);
        const uint8_t* kb = a.k + now.head * L::kRow + chunk * 16;
        const uint8_t* vb = a.v + now.head * L::kRow + chunk * 16;
#pragma unroll
        for (int i = 0; i < kTile; i += kStep) {
          const int r = i + r_lane;
          const int src = __shfl_sync(0xffffffffu, row, r);
          const int64_t off = src < 0 ? 0 : src * row_bytes;
          const uint32_t to = dst + L::at(r, chunk);
          cp16z(to, kb + off, src >= 0);
          cp16z(to + L::kKV, vb + off, src >= 0);
        }
        if constexpr (FP8) {
          const int64_t off = row < 0 ? 0 : static_cast<int64_t>(row) * a.Hkv + now.head;
          const uint32_t to = smem_u32(scales + st * 2 * kTile + lane);
          cp4z(to, a.ks + off, row >= 0);
          cp4z(to + kTile * 4, a.vs + off, row >= 0);
        }
      }
      cp_async_mbar_arrive_noinc(&full[st]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
      now = ahead;
      ahead = later;
      pg = next_pg;
    }
    cp_async_wait_all();
  } else {
    // ============================================================= compute
    const int g = lane >> 2, t = lane & 3;
    // Queries as columns: head g, in the order of d that K is read in (bf16:
    // ldmatrix, words 2 t and 2 t + 8 of 16; fp8: 16 codes a lane and load)
    uint32_t qn[D / 16][2], qf[D / 16][2];
    auto fetch = [&]() {
      const bool used = g < a.G;
      const uint16_t* q = a.q + (static_cast<int64_t>(x.row) * a.Hq + x.head * a.G + (used ? g : 0)) * D;
      if constexpr (!FP8) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qn[kk][0] = *reinterpret_cast<const uint32_t*>(q + kk * 16 + 2 * t);
          qn[kk][1] = *reinterpret_cast<const uint32_t*>(q + kk * 16 + 8 + 2 * t);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 16; kk += 2) {
          const uint4 u = *reinterpret_cast<const uint4*>(q + (kk / 4) * 64 + t * 16 + (kk % 4) * 4);
          qn[kk][0] = u.x;
          qn[kk][1] = u.y;
          qn[kk + 1][0] = u.z;
          qn[kk + 1][1] = u.w;
        }
      }
      if (!used) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) qn[kk][0] = qn[kk][1] = 0;
      }
    };
    // The maximum moves only when it grows by more than 2^kGrow: the weights
    // stay in range and most tiles leave o as it is.  fp8: weights are
    // 2^kLift e^(s - m) * (value scale / 2^base), in f16: 11 bits down to 2^-25
    // of the largest, smaller ones to within 2^-36 of it, and at most 2^15.
    constexpr float kGrow = FP8 ? 4.f : 8.f, kLift = 11.f;
    uint32_t n0 = 0, share = 0;
    // this warp's first tile of a share whose first tile is the CTA's n-th
    auto first_tile = [&](uint32_t n) { return x.t0 + static_cast<int>((warp + kComp - n % kComp) % kComp); };
    bool more = w.next(a, &x), ok = true;
    int tile = 0;
    if (more) {
      tile = first_tile(0);
      if (tile < x.t1) fetch();
    }
    while (ok && more) {
      const int t0 = x.t0, t1 = x.t1, own = tile;
      const bool alone = single(x);
      const int64_t out_row = static_cast<int64_t>(x.row) * a.Hq + x.head * a.G;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][0] = qn[kk][0];
        qf[kk][1] = qn[kk][1];
      }
      more = w.next(a, &x);
      if (more) {
        tile = first_tile(n0 + (t1 - t0));
        if (tile < x.t1) fetch();
      }
      const bool mine = own < t1;
      float c2[2] = {a.c2, a.c2};        // by head 2 t, 2 t + 1
      float o[D / 16][4], m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
      float base = -INFINITY, top = -INFINITY;   // fp8: see scale_base
      if (mine) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        if constexpr (FP8) {
          // the codes are widened to f16, so the queries are f16 too: scaled by
          // a power of two that brings the head's largest to 2^14 .. 2^15 (exact;
          // what falls below f16's range is below 2^-39 of the largest)
          uint32_t mx = 0;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t u = qf[kk][i] & 0x7fff7fffu;
              mx = max(mx, max(u & 0xffffu, u >> 16));
            }
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int e = static_cast<int>(mx >> 7);             // biased exponent
          const int up = e == 0 || e == 255 ? 0 : max(-100, min(100, 127 + 14 - e));
          const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
          const float back = a.c2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
          c2[0] = __shfl_sync(0xffffffffu, back, 8 * t);
          c2[1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qf[kk][i] = pack_f16(__uint_as_float(qf[kk][i] << 16) * f, __uint_as_float(qf[kk][i] & 0xffff0000u) * f);
        }
      }
      bool begun = false;
      float far = INFINITY;              // fp8: the tile's keys of this log2 scale and more are done
      for (int at = own; at < t1;) {
        const uint32_t n = n0 + (at - t0), st = n % S;
        if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (n / S) & 1, err, abort))) {
          ok = false;
          break;
        }
        const uint32_t real = reals[st];
        bool again = false;
        if (real) {
          const uint8_t* stage = stages + st * 2 * L::kKV;
          const uint32_t sk = smem_u32(stage), sv = sk + L::kKV;
          float s[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
          if constexpr (!FP8) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t k4[4];
                ldsm4(k4, sk + L::at(j * 16 + (lane & 15), kk * 2 + (lane >> 4)));
                mma<false>(s[j], k4, qf[kk][0], qf[kk][1]);
              }
          } else {
#pragma unroll
            for (int c4 = 0; c4 < D / 64; ++c4) {
              uint4 u[2][2];
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  u[j][i] = *reinterpret_cast<const uint4*>(stage + L::at(j * 16 + i * 8 + L::key(g), c4 * 4 + t));
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint32_t lo = reinterpret_cast<const uint32_t*>(&u[j][0])[i];
                  const uint32_t hi = reinterpret_cast<const uint32_t*>(&u[j][1])[i];
                  uint32_t k4[4];
                  e4m3x4_to_f16x4(lo, &k4[0], &k4[2]);
                  e4m3x4_to_f16x4(hi, &k4[1], &k4[3]);
                  mma<true>(s[j], k4, qf[c4 * 4 + i][0], qf[c4 * 4 + i][1]);
                }
            }
          }
          // scale, mask and the running maximum; rows g and g + 8 of block j are
          // keys 16 j + key(g) and 8 behind it
          const float* ksc = scales + st * 2 * kTile + L::key(g);
          float lv[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float f0 = 1.f, f1 = 1.f;
            if constexpr (FP8) {
              f0 = ksc[j * 16];
              f1 = ksc[j * 16 + 8];
              lv[2 * j] = __log2f(ksc[kTile + j * 16]);
              lv[2 * j + 1] = __log2f(ksc[kTile + j * 16 + 8]);
            }
            s[j][0] *= c2[0] * f0;
            s[j][1] *= c2[1] * f0;
            s[j][2] *= c2[0] * f1;
            s[j][3] *= c2[1] * f1;
          }
          if (real != 0xffffffffu) {
            const uint32_t bits = real >> L::key(g);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const bool r0 = (bits >> (j * 16)) & 1, r1 = (bits >> (j * 16 + 8)) & 1;
              s[j][0] = r0 ? s[j][0] : -INFINITY;
              s[j][1] = r0 ? s[j][1] : -INFINITY;
              s[j][2] = r1 ? s[j][2] : -INFINITY;
              s[j][3] = r1 ? s[j][3] : -INFINITY;
            }
          }
          float mx[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(fmaxf(s[0][i], s[0][i + 2]), fmaxf(s[1][i], s[1][i + 2]));
#pragma unroll
            for (int d = 4; d < 32; d *= 2) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
          }
          const bool move0 = mx[0] > -INFINITY && (m_run[0] == -INFINITY || mx[0] > m_run[0] + kGrow);
          const bool move1 = mx[1] > -INFINITY && (m_run[1] == -INFINITY || mx[1] > m_run[1] + kGrow);
          bool move = move0 || move1;
          float first = 1.f;              // the sum takes a tile's weights once
          if constexpr (FP8) {
            if (far != INFINITY) {
              first = 0.f;
#pragma unroll
              for (int i = 0; i < 4; ++i) lv[i] = lv[i] < far ? lv[i] : -INFINITY;
            }
            move |= fmaxf(fmaxf(lv[0], lv[1]), fmaxf(lv[2], lv[3])) > base;
            move |= fminf(fminf(lv[0], lv[1]), fminf(lv[2], lv[3])) < base - kSpan;
          }
          if (__any_sync(0xffffffffu, move)) {
            const float m0 = move0 ? mx[0] : m_run[0], m1 = move1 ? mx[1] : m_run[1];
            const float f0 = move0 ? exp2_approx(m_run[0] - m0) : 1.f, f1 = move1 ? exp2_approx(m_run[1] - m1) : 1.f;
            m_run[0] = m0;
            m_run[1] = m1;
            float fe = 1.f;
            if constexpr (FP8) {
              float e = fmaxf(fmaxf(lv[0], lv[1]), fmaxf(lv[2], lv[3]));
#pragma unroll
              for (int d = 4; d < 32; d *= 2) e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, d));
              e = ceilf(e);
              const float b = scale_base(e, base, far == INFINITY, &top);
              if (b != base) fe = pow2(base - b);
              base = b;
              far = scale_rest(e, b);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (lv[i] < far) {      // another pass
                  again |= lv[i] != -INFINITY;
                  lv[i] = -INFINITY;
                }
              again = __any_sync(0xffffffffu, again);
            }
            if (begun) {
              l_run[0] *= f0;
              l_run[1] *= f1;
              const float g0 = f0 * fe, g1 = f1 * fe;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[i][0] *= g0;
                o[i][1] *= g1;
                o[i][2] *= g0;
                o[i][3] *= g1;
              }
            }
          }
          begun = true;
          // a head without a finite score so far: exponents against 0 (all e^-inf = 0)
          const float mu[2] = {m_run[0] == -INFINITY ? 0.f : m_run[0], m_run[1] == -INFINITY ? 0.f : m_run[1]};
          // the weights for the product with v, as two bf16 terms (16 bits; the
          // products have time left: reading bounds) or, fp8, as one f16 (11
          // bits); their sum is taken before that rounding
          const float lift = kLift - (base == -INFINITY ? 0.f : base);
          uint32_t p[2][2], rest[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float x0 = s[j][2 * i] - mu[0], x1 = s[j][2 * i + 1] - mu[1];
              const float e0 = exp2_approx(x0), e1 = exp2_approx(x1);
              l_run[0] = FP8 ? fmaf(e0, first, l_run[0]) : l_run[0] + e0;
              l_run[1] = FP8 ? fmaf(e1, first, l_run[1]) : l_run[1] + e1;
              if constexpr (FP8) {
                const float v0 = lv[2 * j + i] + lift;
                p[j][i] = transposed(pack_f16(exp2_approx(x0 + v0), exp2_approx(x1 + v0)));
              } else {
                const uint32_t top = pack_bf16(e0, e1);
                p[j][i] = transposed(top);
                rest[j][i] = transposed(
                    pack_bf16(e0 - __uint_as_float(top << 16), e1 - __uint_as_float(top & 0xffff0000u)));
              }
            }
          }
          // lane i gives the address of row i of an 8 x 8 block, in the keys' order
          if constexpr (!FP8) {
            const int vr = (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int dd = 0; dd < D / 16; ++dd) {
                uint32_t v4[4];
                ldsm4t(v4, sv + L::at(j * 16 + vr, dd * 2 + vc));
                mma<false>(o[dd], v4, p[j][0], p[j][1]);
                mma<false>(o[dd], v4, rest[j][0], rest[j][1]);
              }
          } else {
            // 16-bit transposed loads bring two neighbouring codes of two keys: row
            // g of product dd is d = 16 dd + 2 g, row g + 8 the next one
            const int vr = (lane & 8) + L::key(lane & 7);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t b[4];
                ldsm4t(b, sv + L::at(j * 16 + vr, cc * 2 + (lane >> 4)));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  uint32_t v4[4];
                  e4m3x4_to_f16x4(__byte_perm(b[2 * i], 0, 0x3120), &v4[0], &v4[1]);
                  e4m3x4_to_f16x4(__byte_perm(b[2 * i + 1], 0, 0x3120), &v4[2], &v4[3]);
                  mma<true>(o[cc * 2 + i], v4, p[j][0], p[j][1]);
                }
              }
          }
        }
        if (FP8 && again) continue;
        far = INFINITY;
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        at += kComp;
      }
      if (!ok) break;
      n0 += t1 - t0;
      if (begun) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], d);
      }
      const float unlift = !FP8 ? 1.f : (base == -INFINITY ? 0.f : exp2_approx(base - kLift));
      if (alone) {
        if (mine) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int h = 2 * t + i;
            if (h >= a.G) continue;
            const float inv = l_run[i] == 0.f ? 0.f : unlift / l_run[i];
            uint16_t* to = a.out + (out_row + h) * D;
#pragma unroll
            for (int dd = 0; dd < D / 16; ++dd) {
              // (a head whose scores are all -inf is zero whatever the values hold)
              const uint32_t y = begun && l_run[i] != 0.f ? pack_bf16(o[dd][i] * inv, o[dd][2 + i] * inv) : 0;
              if constexpr (!FP8) {
                to[dd * 16 + g] = static_cast<uint16_t>(y & 0xffff);
                to[dd * 16 + 8 + g] = static_cast<uint16_t>(y >> 16);
              } else {
                *reinterpret_cast<uint32_t*>(to + dd * 16 + 2 * g) = y;
              }
            }
            if (a.lse && g == 0)
              a.lse[out_row + h] = l_run[i] == 0.f ? -INFINITY : (m_run[i] + log2f(l_run[i])) * kLn2;
          }
        }
        continue;
      }
      // this warp's state of the row
      const uint32_t buf = share & 1;
      if (share >= 2 && !__all_sync(0xffffffffu, mbar_wait(&st_free[buf], ((share >> 1) - 1) & 1, err, abort))) break;
      float* to = states + buf * L::kStates + warp * 8 * L::kState;
      if (begun) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* h = to + (2 * t + i) * L::kState;
#pragma unroll
          for (int dd = 0; dd < D / 16; ++dd) {
            if constexpr (!FP8) {
              h[dd * 16 + g] = o[dd][i];
              h[dd * 16 + 8 + g] = o[dd][2 + i];
            } else {
              *reinterpret_cast<float2*>(h + dd * 16 + 2 * g) = make_float2(o[dd][i] * unlift, o[dd][2 + i] * unlift);
            }
          }
        }
      }
      if (g == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *reinterpret_cast<float2*>(to + (2 * t + i) * L::kState + D) = make_float2(m_run[i], l_run[i]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&st_full[buf]);
      ++share;
    }
  }
}

template <int D, bool FP8>
cudaError_t launch_few(const RowsArgs& a, int grid, cudaStream_t st) {
  using L = Few<D, FP8>;
  static ReadyOnce ready;
  const cudaError_t e = ready.shared_memory(k_attend_few<D, FP8>, L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_after(k_attend_few<D, FP8>, dim3(grid), dim3(L::kThreads), L::kBytes, st, a);
}

}  // namespace

int rows_few_tile() { return kTile; }

cudaError_t launch_rows_few(const RowsArgs& a, int D, bool fp8, int grid, cudaStream_t st) {
  if (D == 64) return fp8 ? launch_few<64, true>(a, grid, st) : launch_few<64, false>(a, grid, st);
  return fp8 ? launch_few<128, true>(a, grid, st) : launch_few<128, false>(a, grid, st);
}

}  // namespace aiidx
