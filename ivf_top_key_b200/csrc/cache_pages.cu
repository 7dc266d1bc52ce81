// Pages of a key-value cache: extend, write, fork, free, compact.
//
// Page tables, lengths and reference counts live in device memory and every
// change to them is made by a kernel in stream order, so a decode step that
// takes pages, writes its token and attends can be captured in a CUDA graph
// and replayed.  Allocation is deterministic: the lowest free pages, in the
// order of the call's list.
//
// Pages that hold more than one sequence's tokens are full (a fork copies the
// part page), and a write that would reach one is refused, so a page is written
// only while one sequence owns it.
//
// What bounds them: a call is one CTA that plans (a scan of a thousand reference
// counts takes about 4 us) and a grid that moves pages at the copy rate of HBM: 226
// pages of 4 layers (474 MB read and written) 80 us, 5.9 TB/s.  An extend looks
// for repeated sequences along the list and gives a sequence's pages by one thread:
// with their release 8 sequences by one token take 5 us, 1024 64 us, one sequence
// by 8192 pages 440 us.  A write is a warp per token and head, bound by its chain
// of look-ups: 8192 tokens of 8 heads of 128 (67 MB read and written) 20 us, fp8
// 35 us (quantising), 256 tokens 5 us.
#include <mutex>

#include "../../include/ai_index.h"
#include "common.cuh"
#include "kernels.h"

namespace aiidx {
namespace {

constexpr int kPlan = 1024;  // threads of the planning CTA

int fail(int code, const char* msg) {
  set_last_error(msg);
  return code;
}

// Device view of a cache.
struct View {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t page_bytes;    // K (or V) bytes of a page of one layer
  int slot_bytes;        // of one token
  int scale_floats;      // scales of one token (fp8), else 0
  int n_layers, n_pages, page_size;
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int n_seqs, width;
  int32_t* status;
};

__device__ __forceinline__ void flag(const View& c, int bit) {
  atomicOr(c.status, bit);
}
__device__ __forceinline__ bool listed_before(const int32_t* list, int i) {
  for (int j = 0; j < i; ++j)
    if (list[j] == list[i]) return true;
  return false;
}

// Exclusive prefix of one int per thread of the planning CTA.
__device__ int plan_scan(int x, int* total, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  *total = sums[kPlan / 32 - 1];
  return (warp ? sums[warp - 1] : 0) + inc - x;
}

// The `want` lowest free pages in ascending order to list; returns how many
// there are (at most want).  Called by the whole planning CTA.
__device__ int lowest_free(const View& c, int want, int32_t* list, int* sums) {
  int found = 0;
  for (int p0 = 0; p0 < c.n_pages && found < want; p0 += 4 * kPlan) {
    const int p = p0 + 4 * static_cast<int>(threadIdx.x);
    int f[4], n = 0;
    for (int i = 0; i < 4; ++i) {
      f[i] = p + i < c.n_pages && c.refs[p + i] <= 0;
      n += f[i];
    }
    int total;
    int at = found + plan_scan(n, &total, sums);
    for (int i = 0; i < 4; ++i)
      if (f[i]) {
        if (at < want) list[at] = p + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return found < want ? found : want;
}

// ------------------------------------------------------------------- extend
// Two passes over the list: pages each sequence needs with their prefix,
// then the assignment.  scratch: [n] first page rank (-1: refused, -2: more
// pages than the cache has), then the free pages.
__global__ void __launch_bounds__(kPlan) k_extend(View c, const int32_t* seqs, const int32_t* counts, int n,
                                                  int32_t* scratch) {
  __shared__ int sums[32];
  dependency_wait();
  int32_t* rank = scratch;
  int32_t* fresh = scratch + n;
  int64_t before = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int need = 0, ok = 0;
    if (i < n) {
      const int s = seqs[i], add = counts[i];
      if (s < 0 || s >= c.n_seqs || add < 0 || c.lens[s] < 0 || listed_before(seqs, i)) {
        flag(c, AI_DEVFLAG_RANGE);
      } else {
        const int64_t len = c.lens[s], end = len + add;
        if (end > static_cast<int64_t>(c.width) * c.page_size) {
          flag(c, AI_DEVFLAG_CAPACITY);
        } else {
          ok = 1;
          need = static_cast<int>((end + c.page_size - 1) / c.page_size - (len + c.page_size - 1) / c.page_size);
          need = min(need, c.n_pages + 1);  // the prefixes of a pass stay below 2^31 (n_pages <= 2^20)
        }
      }
    }
    // a prefix beyond the cache's pages stays beyond them: 64 bits, clamped
    const int most = c.n_pages + 1;
    int total;
    const int p = plan_scan(need, &total, sums);
    if (i < n) {
      const int64_t at = before + p;
      // an entry that needs no page is lengthened whatever the ones before it ask for
      rank[i] = !ok ? -1 : (need > 0 && at + need > c.n_pages ? -2 : static_cast<int>(at));
    }
    before = before + total > most ? most : before + total;
  }
  __syncthreads();
  const int want = before > c.n_pages ? c.n_pages : static_cast<int>(before);
  const int have = lowest_free(c, want, fresh, sums);
  for (int i = threadIdx.x; i < n; i += kPlan) {
    if (rank[i] == -1) continue;
    const int s = seqs[i];
    const int64_t len = c.lens[s], end = len + counts[i];   // (below 2^31, rounded up maybe not)
    const int p0 = static_cast<int>((len + c.page_size - 1) / c.page_size);
    const int p1 = static_cast<int>((end + c.page_size - 1) / c.page_size);
    if (rank[i] < 0 || (p1 > p0 && rank[i] + (p1 - p0) > have)) {
      flag(c, AI_DEVFLAG_CAPACITY);
      continue;
    }
    for (int p = p0; p < p1; ++p) {
      const int page = fresh[rank[i] + p - p0];
      c.tables[static_cast<int64_t>(s) * c.width + p] = page;
      c.refs[page] = 1;
    }
    c.lens[s] = static_cast<int>(end);
  }
}

// -------------------------------------------------------------------- write
// One warp per (token, head) row of K and of V.  Pages that several sequences
// hold are the first ones of their rows (a fork shares all full pages), so a
// segment whose first page is one sequence's reaches no shared one; the token's
// own page is looked at too, for tables that were made otherwise.
template <bool FP8>
__global__ void k_write(View c, int64_t layer_slots, int layer, const uint16_t* kn, const uint16_t* vn,
                        const int32_t* seqs, const int32_t* cu, int n, int n_tokens, int Hkv, int D) {
  dependency_wait();
  const int64_t wid = (blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= static_cast<int64_t>(n_tokens) * Hkv) return;
  const int tok = static_cast<int>(wid / Hkv), h = static_cast<int>(wid % Hkv);
  if (tok < cu[0] || tok >= cu[n]) return;
  int lo = 0, hi = n;  // the segment: cu[lo] <= tok < cu[lo + 1]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= tok) lo = mid;
    else hi = mid;
  }
  const int s = seqs[lo];
  bool again = false;
  for (int j = lane; j < lo; j += 32) again |= seqs[j] == s && cu[j + 1] > cu[j];
  if (__any_sync(0xffffffffu, again) || s < 0 || s >= c.n_seqs) {
    if (lane == 0) flag(c, AI_DEVFLAG_RANGE);
    return;
  }
  const int len = c.lens[s];
  const int64_t pos = static_cast<int64_t>(len) - (cu[lo + 1] - tok);
  const int64_t first = static_cast<int64_t>(len) - (cu[lo + 1] - cu[lo]);
  // lane 0 looks up the token's page, lane 1 the segment's first one
  const int64_t at = lane == 1 ? max(first, static_cast<int64_t>(0)) : pos;
  int page = -1;
  bool shared = false;
  if (lane < 2 && at >= 0 && at < static_cast<int64_t>(c.width) * c.page_size) {
    page = c.tables[static_cast<int64_t>(s) * c.width + static_cast<uint32_t>(at) / static_cast<uint32_t>(c.page_size)];
    if (page < 0 || page >= c.n_pages) page = -1;
    else if (c.refs) shared = c.refs[page] > 1;
  }
  page = __shfl_sync(0xffffffffu, page, 0);
  if (__any_sync(0xffffffffu, shared) || page < 0) {
    if (lane == 0) flag(c, AI_DEVFLAG_RANGE);
    return;
  }
  // a lane's first words of both rows at once
  const int64_t src = (static_cast<int64_t>(tok) * Hkv + h) * D;
  uint32_t head[2][2];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      head[which][u] = lane + 32 * u < D / 2 ? reinterpret_cast<const uint32_t*>((which ? vn : kn) + src)[lane + 32 * u] : 0;
  const int slot = static_cast<int>(static_cast<uint32_t>(pos) % static_cast<uint32_t>(c.page_size));
  const int64_t row = (layer * layer_slots + static_cast<int64_t>(page) * c.page_size + slot) * Hkv + h;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>((which ? vn : kn) + src);
    auto word = [&](int i) { return i < 32 ? head[which][0] : (i < 64 ? head[which][1] : x[i]); };
    uint8_t* dst = which ? c.v : c.k;
    if constexpr (!FP8) {
      uint32_t* y = reinterpret_cast<uint32_t*>(dst + row * D * 2);
      for (int i = lane; i < D / 2; i += 32) y[i] = word(i);
    } else {
      // scale amax / 448 and e4m3 codes of the row, as for fp8 key stores
      float amax = 0.f;
      for (int i = lane; i < D / 2; i += 32) {
        const uint32_t u = word(i);
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u << 16)), fabsf(__uint_as_float(u & 0xffff0000u))));
      }
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      uint16_t* y = reinterpret_cast<uint16_t*>(dst + row * D);
      for (int i = lane; i < D / 2; i += 32) {
        const uint32_t u = word(i);
        const uint16_t a = __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(u << 16), scale), __NV_SATFINITE, __NV_E4M3);
        const uint16_t b =
            __nv_cvt_float_to_fp8(__fdiv_rn(__uint_as_float(u & 0xffff0000u), scale), __NV_SATFINITE, __NV_E4M3);
        y[i] = static_cast<uint16_t>(a | (b << 8));
      }
      if (lane == 0) (which ? c.vs : c.ks)[row] = scale;
    }
  }
}

// --------------------------------------------------------------------- fork
// All forks read the state before the call.  plan[i]: the fresh page of fork
// i's part page, -1 where it has none, -2 where the fork is refused; length[i]:
// the source's length.  What the new sequences own alone is written at once (a
// source that is another fork's target was empty, so its row is not read).
__global__ void __launch_bounds__(kPlan) k_fork_plan(View c, const int32_t* src, const int32_t* dst, int n,
                                                     int32_t* plan, int32_t* length, int32_t* fresh) {
  __shared__ int sums[32];
  dependency_wait();
  int before = 0;
  for (int i0 = 0; i0 < n; i0 += kPlan) {
    const int i = i0 + threadIdx.x;
    int need = 0, code = -2;
    if (i < n) {
      const int a = src[i], b = dst[i];
      if (a < 0 || a >= c.n_seqs || b < 0 || b >= c.n_seqs || c.lens[b] != 0 || listed_before(dst, i) ||
          c.lens[a] < 0 || c.lens[a] > static_cast<int64_t>(c.width) * c.page_size) {
        flag(c, AI_DEVFLAG_RANGE);
      } else {
        length[i] = c.lens[a];
        need = length[i] % c.page_size != 0;
        code = -1;
      }
    }
    int total;
    const int p = plan_scan(need, &total, sums);
    if (i < n) plan[i] = need ? before + p : code;
    before += total;
  }
  __syncthreads();
  const int have = lowest_free(c, before < c.n_pages ? before : c.n_pages, fresh, sums);
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int rank = plan[i];
    if (rank >= have) {
      plan[i] = -2;
      flag(c, AI_DEVFLAG_CAPACITY);
    } else if (rank != -2) {
      if (rank >= 0) {
        plan[i] = fresh[rank];
        c.tables[static_cast<int64_t>(dst[i]) * c.width + length[i] / c.page_size] = fresh[rank];
        c.refs[fresh[rank]] = 1;
      }
      c.lens[dst[i]] = length[i];
    }
  }
}

// Copies chunk `chunk` of the first `slots` tokens of a page of one layer: K
// and V bytes as one run of 16-byte units, kUnits of them a thread, all loaded
// before the first is stored; scales with chunk 0.  A chunk is 8 KB: 16 blocks
// an SM keep 128 KB of loads under way (with a page's 16 KB parts of K, then V,
// to a block, 64 forks of 16 layers and their release took 84 us, now 71).
constexpr int kMoveThreads = 128, kUnits = 4;
__host__ __device__ constexpr int64_t chunks_of(int64_t bytes) {
  return (2 * bytes / 16 + kMoveThreads * kUnits - 1) / (kMoveThreads * kUnits);
}
__device__ __forceinline__ void copy_chunk(const View& c, int layer, int from, int to, int slots, int64_t chunk) {
  const int64_t l = static_cast<int64_t>(layer) * c.n_pages;
  const int64_t n = static_cast<int64_t>(slots) * c.slot_bytes / 16;  // units of K, and of V
  const int64_t src = (l + from) * c.page_bytes, dst = (l + to) * c.page_bytes;
  const int64_t u0 = chunk * (kMoveThreads * kUnits) + threadIdx.x;
  uint4 x[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = u0 + i * kMoveThreads;
    if (u < 2 * n) x[i] = *reinterpret_cast<const uint4*>((u < n ? c.k + u * 16 : c.v + (u - n) * 16) + src);
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int64_t u = u0 + i * kMoveThreads;
    if (u < 2 * n) *reinterpret_cast<uint4*>((u < n ? c.k + u * 16 : c.v + (u - n) * 16) + dst) = x[i];
  }
  if (chunk == 0 && c.scale_floats) {
    const int64_t ps = static_cast<int64_t>(c.page_size) * c.scale_floats;
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(slots) * c.scale_floats; i += kMoveThreads) {
      c.ks[(l + to) * ps + i] = c.ks[(l + from) * ps + i];
      c.vs[(l + to) * ps + i] = c.vs[(l + from) * ps + i];
    }
  }
}

// grid (chunks of a page, layers, forks): the filled slots of the part page,
// and the row's full pages, which gain a holder.
__global__ void __launch_bounds__(kMoveThreads) k_fork_move(View c, const int32_t* src, const int32_t* dst,
                                                            const int32_t* plan, const int32_t* length, int n) {
  dependency_wait();
  for (int i = blockIdx.z; i < n; i += gridDim.z) {
    const int fresh = plan[i];
    if (fresh == -2) continue;
    const int len = length[i];
    const int full = len / c.page_size, slots = len % c.page_size;
    const int32_t* from = c.tables + static_cast<int64_t>(src[i]) * c.width;
    if (fresh >= 0) {
      const int old = from[full];
      if (old >= 0 && old < c.n_pages) {
        const int64_t used = chunks_of(static_cast<int64_t>(slots) * c.slot_bytes);
        for (int layer = blockIdx.y; layer < c.n_layers; layer += gridDim.y)
          for (int64_t chunk = blockIdx.x; chunk < used; chunk += gridDim.x) copy_chunk(c, layer, old, fresh, slots, chunk);
      } else {
        flag(c, AI_DEVFLAG_RANGE);
      }
    }
    if (blockIdx.y == 0) {
      int32_t* to = c.tables + static_cast<int64_t>(dst[i]) * c.width;
      for (int p = blockIdx.x * kMoveThreads + threadIdx.x; p < full; p += gridDim.x * kMoveThreads) {
        const int page = from[p];
        to[p] = page;
        if (page >= 0 && page < c.n_pages) atomicAdd(c.refs + page, 1);
        else flag(c, AI_DEVFLAG_RANGE);
      }
    }
  }
}

// --------------------------------------------------------------------- free
// One block per listed sequence; the block that takes the length owns it, so
// a sequence listed twice is released once.
__global__ void __launch_bounds__(256) k_free(View c, const int32_t* seqs, int n) {
  __shared__ int sh_len;
  dependency_wait();
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = seqs[i];
    __syncthreads();
    if (threadIdx.x == 0) {
      sh_len = 0;
      if (s >= 0 && s < c.n_seqs) sh_len = atomicExch(c.lens + s, 0);
      else flag(c, AI_DEVFLAG_RANGE);
    }
    __syncthreads();
    const int64_t used = (static_cast<int64_t>(sh_len) + c.page_size - 1) / c.page_size;
    for (int64_t p = threadIdx.x; p < used && p < c.width; p += blockDim.x) {
      int32_t* e = c.tables + static_cast<int64_t>(s) * c.width + p;
      const int page = *e;
      *e = -1;
      if (page >= 0 && page < c.n_pages) atomicSub(c.refs + page, 1);
      else flag(c, AI_DEVFLAG_RANGE);
    }
  }
}

// ------------------------------------------------------------------ compact
// With L live pages, the i-th live page at or behind L moves to the i-th free
// page before L: as many moves as there are holes, sources and targets apart,
// so the pages move in parallel.  scratch: map [n_pages] (-1: stays), from
// [n_pages], to [n_pages], count.
__global__ void __launch_bounds__(kPlan) k_compact_plan(View c, int32_t* map, int32_t* from, int32_t* to,
                                                        int32_t* count) {
  __shared__ int sums[32];
  dependency_wait();
  int live = 0;
  for (int p = threadIdx.x; p < c.n_pages; p += kPlan) live += c.refs[p] > 0;
  int n_live;
  plan_scan(live, &n_live, sums);
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < c.n_pages; p0 += kPlan) {
    const int p = p0 + threadIdx.x;
    const bool in = p < c.n_pages;
    const int r = in ? c.refs[p] : 0;
    const int hole = in && p < n_live && r <= 0, move = in && p >= n_live && r > 0;
    int n;
    const int at = (p0 < n_live ? plan_scan(hole, &n, sums) : 0);
    if (p0 < n_live) {
      if (hole) to[holes + at] = p;
      holes += n;
    }
    int nm = 0;
    if (p0 + kPlan > n_live) {
      const int am = plan_scan(move, &nm, sums);
      if (move) from[movers + am] = p;
    }
    movers += nm;
    if (in) map[p] = -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kPlan) map[from[i]] = to[i];
  if (threadIdx.x == 0) *count = movers;
}

__global__ void __launch_bounds__(kMoveThreads) k_compact_move(View c, const int32_t* map, const int32_t* from,
                                                               const int32_t* to, const int32_t* count) {
  dependency_wait();
  const int n = *count;
  const int64_t chunks = chunks_of(c.page_bytes), units = static_cast<int64_t>(n) * c.n_layers * chunks;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t page = u / chunks, chunk = u - page * chunks;
    const int i = static_cast<int>(page / c.n_layers), layer = static_cast<int>(page - static_cast<int64_t>(i) * c.n_layers);
    copy_chunk(c, layer, from[i], to[i], c.page_size, chunk);
    if (layer == 0 && chunk == 0 && threadIdx.x == 0) {
      c.refs[to[i]] = c.refs[from[i]];
      c.refs[from[i]] = 0;
    }
  }
  // the tables follow
  const int64_t entries = static_cast<int64_t>(c.n_seqs) * c.width;
  for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < entries;
       e += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int page = c.tables[e];
    if (page >= 0 && page < c.n_pages && map[page] >= 0) c.tables[e] = map[page];
  }
}

// Where flags go when the caller gives no status word, and what the last read
// took from there.
__device__ int32_t g_status[2];

__global__ void k_take_status() {
  dependency_wait();
  g_status[1] = atomicExch(&g_status[0], 0);
}

View view_of(const ai_cache* c) {
  View v{};
  const int es = c->dtype == AI_BF16 ? 2 : 1;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.ks = c->k_scale;
  v.vs = c->v_scale;
  v.slot_bytes = c->n_kv_heads * c->head_dim * es;
  v.page_bytes = static_cast<int64_t>(v.slot_bytes) * c->page_size;
  v.scale_floats = es == 1 ? c->n_kv_heads : 0;
  v.n_layers = c->n_layers;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.tables = c->tables;
  v.lens = c->lens;
  v.refs = c->refs;
  v.n_seqs = c->n_seqs;
  v.width = c->max_pages;
  v.status = c->status ? c->status : default_status();
  return v;
}

int no_status() { return fail(AI_ERR_CUDA, "the device's status word was not found"); }
int done(cudaError_t e) { return e == cudaSuccess ? AI_OK : fail(AI_ERR_CUDA, cudaGetErrorString(e)); }

int check_tables(const ai_cache* c) {
  if (!c) return fail(AI_ERR_ARG, "null cache");
  if (!c->tables || !c->lens) return fail(AI_ERR_ARG, "null tables or lens");
  if (c->n_pages <= 0 || c->page_size <= 0 || c->n_seqs <= 0 || c->max_pages <= 0)
    return fail(AI_ERR_ARG, "page and sequence counts must be positive");
  if (c->n_pages > (1 << 20)) return fail(AI_ERR_ARG, "more than 2^20 pages");
  if (static_cast<int64_t>(c->n_pages) * c->page_size > 0x7fffffff ||
      static_cast<int64_t>(c->max_pages) * c->page_size > 0x7fffffff)
    return fail(AI_ERR_ARG, "token slots beyond 2^31 - 1");
  return AI_OK;
}

int check_list(const ai_cache* c, const void* list, int32_t n) {
  if (!c->refs) return fail(AI_ERR_ARG, "null refs");
  if (n < 0 || (n > 0 && !list)) return fail(AI_ERR_ARG, "bad list");
  return AI_OK;
}

}  // namespace

int device_sms() {
  static std::atomic<int> known[kMaxDevices] = {};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) return 148;
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

int32_t* default_status() {
  static std::atomic<int32_t*> known[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  int32_t* p = known[dev].load(std::memory_order_relaxed);
  if (!p) {
    void* at = nullptr;
    if (cudaGetSymbolAddress(&at, g_status) != cudaSuccess) return nullptr;
    p = static_cast<int32_t*>(at);
    known[dev].store(p, std::memory_order_relaxed);
  }
  return p;
}

cudaError_t ReadyOnce::allow(const void* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

int check_cache(const ai_cache* c) {
  const int rc = check_tables(c);
  if (rc) return rc;
  if (!c->k || !c->v) return fail(AI_ERR_ARG, "null pages");
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) % 16 != 0)
    return fail(AI_ERR_ARG, "pages must be 16-byte aligned");
  if (c->dtype != AI_BF16 && c->dtype != AI_FP8E4M3) return fail(AI_ERR_ARG, "the cache holds bf16 or fp8 e4m3");
  if ((c->dtype == AI_FP8E4M3) != (c->k_scale != nullptr) || (c->dtype == AI_FP8E4M3) != (c->v_scale != nullptr))
    return fail(AI_ERR_ARG, "k_scale and v_scale go with an fp8 cache, and only with one");
  if (c->n_layers <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->head_dim % 16 != 0 || c->head_dim > 1024)
    return fail(AI_ERR_ARG, "layers and heads must be positive, head_dim a multiple of 16 up to 1024");
  return AI_OK;
}

}  // namespace aiidx

extern "C" int ai_cache_workspace(const ai_cache* c, int32_t n, int64_t* bytes_out) {
  using namespace aiidx;
  if (!c || !bytes_out || n < 0 || c->n_pages <= 0) return fail(AI_ERR_ARG, "bad cache, list length or null output");
  *bytes_out = (3 * static_cast<int64_t>(c->n_pages) + 2 * static_cast<int64_t>(n) + 4) * 4;
  return AI_OK;
}

// The workspace holds what ai_cache_workspace says for this call.
static int check_ws(const ai_cache* c, int32_t n, const void* ws, int64_t bytes) {
  int64_t need = 0;
  const int rc = ai_cache_workspace(c, n, &need);
  if (rc) return rc;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 4 != 0 || bytes < need)
    return aiidx::fail(AI_ERR_ARG, "workspace too small or misaligned");
  return AI_OK;
}

extern "C" int ai_cache_extend(const ai_cache* c, const int32_t* seqs_dev, const int32_t* counts_dev, int32_t n,
                               void* workspace_dev, int64_t workspace_bytes, void* cuda_stream) {
  using namespace aiidx;
  int rc = check_tables(c);
  if (!rc) rc = check_list(c, seqs_dev, n);
  if (!rc && n > 0 && !counts_dev) rc = fail(AI_ERR_ARG, "null counts");
  if (!rc) rc = check_ws(c, n, workspace_dev, workspace_bytes);
  if (rc || n == 0) return rc;
  const View v = view_of(c);
  if (!v.status) return no_status();
  return done(launch_after(k_extend, dim3(1), dim3(kPlan), 0, static_cast<cudaStream_t>(cuda_stream), v, seqs_dev, counts_dev,
                           n, static_cast<int32_t*>(workspace_dev)));
}

extern "C" int ai_cache_write(const ai_cache* c, int32_t layer, const void* k_dev, const void* v_dev,
                              const int32_t* seqs_dev, const int32_t* cu_dev, int32_t n, int32_t n_tokens,
                              void* cuda_stream) {
  using namespace aiidx;
  int rc = check_cache(c);
  if (rc) return rc;
  if (layer < 0 || layer >= c->n_layers) return fail(AI_ERR_ARG, "layer out of range");
  if (n < 0 || n_tokens < 0) return fail(AI_ERR_ARG, "negative list length or token count");
  if (n == 0 || n_tokens == 0) return AI_OK;
  if (!k_dev || !v_dev || !seqs_dev || !cu_dev) return fail(AI_ERR_ARG, "null pointer argument");
  if ((reinterpret_cast<uintptr_t>(k_dev) | reinterpret_cast<uintptr_t>(v_dev)) % 4 != 0)
    return fail(AI_ERR_ARG, "new keys and values must be 4-byte aligned");
  const int64_t blocks = (static_cast<int64_t>(n_tokens) * c->n_kv_heads * 32 + 255) / 256;
  if (blocks > 0x7fffffff) return fail(AI_ERR_ARG, "too many tokens");
  const int64_t slots = static_cast<int64_t>(c->n_pages) * c->page_size;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const uint16_t* kn = static_cast<const uint16_t*>(k_dev);
  const uint16_t* vn = static_cast<const uint16_t*>(v_dev);
  const dim3 grid(static_cast<unsigned>(blocks));
  const View v = view_of(c);
  if (!v.status) return no_status();
  return done(c->dtype == AI_BF16
                  ? launch_after(k_write<false>, grid, dim3(256), 0, st, v, slots, layer, kn, vn, seqs_dev, cu_dev, n,
                                 n_tokens, c->n_kv_heads, c->head_dim)
                  : launch_after(k_write<true>, grid, dim3(256), 0, st, v, slots, layer, kn, vn, seqs_dev, cu_dev, n,
                                 n_tokens, c->n_kv_heads, c->head_dim));
}

extern "C" int ai_cache_fork(const ai_cache* c, const int32_t* src_dev, const int32_t* dst_dev, int32_t n,
                             void* workspace_dev, int64_t workspace_bytes, void* cuda_stream) {
  using namespace aiidx;
  int rc = check_cache(c);
  if (!rc) rc = check_list(c, src_dev, n);
  if (!rc && n > 0 && !dst_dev) rc = fail(AI_ERR_ARG, "null dst");
  if (!rc) rc = check_ws(c, n, workspace_dev, workspace_bytes);
  if (rc || n == 0) return rc;
  const View v = view_of(c);
  if (!v.status) return no_status();
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  int32_t* plan = static_cast<int32_t*>(workspace_dev);
  int32_t* length = plan + n;
  int32_t* fresh = length + n;
  const int64_t chunks = chunks_of(v.page_bytes);
  const dim3 grid(static_cast<unsigned>(chunks < 256 ? chunks : 256), v.n_layers < 1024 ? v.n_layers : 1024,
                  n < 1024 ? n : 1024);
  rc = done(launch_after(k_fork_plan, dim3(1), dim3(kPlan), 0, st, v, src_dev, dst_dev, n, plan, length, fresh));
  if (rc) return rc;
  return done(launch_after(k_fork_move, grid, dim3(kMoveThreads), 0, st, v, src_dev, dst_dev, plan, length, n));
}

extern "C" int ai_cache_free(const ai_cache* c, const int32_t* seqs_dev, int32_t n, void* cuda_stream) {
  using namespace aiidx;
  int rc = check_tables(c);
  if (!rc) rc = check_list(c, seqs_dev, n);
  if (rc || n == 0) return rc;
  const View v = view_of(c);
  if (!v.status) return no_status();
  return done(launch_after(k_free, dim3(n < 4096 ? n : 4096), dim3(256), 0, static_cast<cudaStream_t>(cuda_stream), v,
                           seqs_dev, n));
}

extern "C" int ai_cache_compact(const ai_cache* c, void* workspace_dev, int64_t workspace_bytes, void* cuda_stream) {
  using namespace aiidx;
  int rc = check_cache(c);
  if (!rc) rc = check_list(c, nullptr, 0);
  if (!rc) rc = check_ws(c, 0, workspace_dev, workspace_bytes);
  if (rc) return rc;
  const View v = view_of(c);
  if (!v.status) return no_status();
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  int32_t* map = static_cast<int32_t*>(workspace_dev);
  int32_t* from = map + c->n_pages;
  int32_t* to = from + c->n_pages;
  int32_t* count = to + c->n_pages;
  rc = done(launch_after(k_compact_plan, dim3(1), dim3(kPlan), 0, st, v, map, from, to, count));
  if (rc) return rc;
  return done(launch_after(k_compact_move, dim3(16 * device_sms()), dim3(kMoveThreads), 0, st, v, map, from, to, count));
}

extern "C" int ai_status_read(int32_t* bits_out, void* cuda_stream) {
  using namespace aiidx;
  if (!bits_out) return fail(AI_ERR_ARG, "null output");
  static std::mutex one;   // g_status[1] is one reader's at a time
  std::lock_guard<std::mutex> lock(one);
  const int32_t* word = default_status();
  if (!word) return no_status();
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = launch_after(k_take_status, dim3(1), dim3(1), 0, st);
  if (e == cudaSuccess) e = cudaMemcpyAsync(bits_out, word + 1, sizeof(int32_t), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return done(e);
}
