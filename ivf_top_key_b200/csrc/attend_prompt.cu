// Causal attention over packed prompts, grouped heads.
//
//   o_i = sum_{j <= i + Lk - Lq} e^(s_ij - m_i) v_j / sum_j e^(s_ij - m_i)
//
// One warp per (query, head): lanes hold 32 keys' scores at a time, the
// running maximum and sum in fp32, and the output spread over the lanes.
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
  if (!ok && a.status) atomicOr(a.status, AI_DEVFLAG_RANGE);
  return ok;
}

// One query row of one head by one warp, reading only the keys it sees.
template <int D>
__device__ void attend_row(const PromptArgs& a, int qi, int h, int k0, int n_keys, float* sq /* [D] of this warp */) {
  const int lane = threadIdx.x & 31;
  const uint16_t* q = a.q + qi * a.q_tok + h * a.q_head;
  __syncwarp();
  for (int d = lane; d < D; d += 32) sq[d] = bf16_bits_to_f32(q[d]);
  __syncwarp();
  const int kh = h / a.G;
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < n_keys; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < n_keys) {
      const uint16_t* k = a.k + static_cast<int64_t>(k0 + j) * a.k_tok + kh * a.k_head;
      float x = 0.f;
      for (int d = 0; d < D; d += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(k + d);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x = fmaf(sq[d + 2 * i], __uint_as_float(w[i] << 16), x);
          x = fmaf(sq[d + 2 * i + 1], __uint_as_float(w[i] & 0xffff0000u), x);
        }
      }
      s = x * a.c2;
    }
    float mx = s;
    for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
    const float mn = fmaxf(m, mx), mz = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - mz), p = exp2f(s - mz);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
    const int n = min(32, n_keys - j0);
    for (int jj = 0; jj < n; ++jj) {
      const float pj = __shfl_sync(0xffffffffu, p, jj);
      const uint16_t* v = a.v + static_cast<int64_t>(k0 + j0 + jj) * a.v_tok + kh * a.v_head;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pj, bf16_bits_to_f32(v[i * 32 + lane]), o[i]);
    }
  }
  for (int i = 16; i > 0; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
  uint16_t* out = a.out + (static_cast<int64_t>(qi) * a.Hq + h) * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const __nv_bfloat16 b = __float2bfloat16_rn(l == 0.f ? 0.f : o[i] / l);
    out[i * 32 + lane] = *reinterpret_cast<const uint16_t*>(&b);
  }
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(qi) * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
__global__ void __launch_bounds__(256) k_prompt_rows(PromptArgs a) {
  __shared__ float sq[8][D];
  const int warp = threadIdx.x >> 5;
  const int b = blockIdx.y;
  int q0, lq, k0, lk;
  if (!seq_rows(a, b, &q0, &lq, &k0, &lk)) return;
  const int64_t n = static_cast<int64_t>(lq) * a.Hq;
  for (int64_t i = blockIdx.x * 8ll + warp; i < n; i += gridDim.x * 8ll) {
    const int row = static_cast<int>(i / a.Hq), h = static_cast<int>(i % a.Hq);
    const int64_t seen = static_cast<int64_t>(lk) - lq + row + 1;
    attend_row<D>(a, q0 + row, h, k0, seen < 0 ? 0 : static_cast<int>(seen), sq[warp]);
  }
}

}  // namespace
}  // namespace aiidx

extern "C" int ai_attend_prompt(const void* q_dev, const int64_t* q_strides, const void* k_dev,
                                const int64_t* k_strides, const void* v_dev, const int64_t* v_strides,
                                const int32_t* cu_q_dev, const int32_t* cu_k_dev, int32_t n_seqs, int32_t total_q,
                                int32_t total_k, int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, float scale,
                                void* out_dev, float* lse_dev, int32_t* status_dev, void* cuda_stream) {
  using namespace aiidx;
  if (!q_strides || !k_strides || !v_strides || !cu_q_dev || !cu_k_dev) return fail(AI_ERR_ARG, "null pointer argument");
  if (n_seqs < 0 || total_q < 0 || total_k < 0) return fail(AI_ERR_ARG, "negative sequence or token count");
  if ((total_q > 0 && (!q_dev || !out_dev)) || (total_k > 0 && (!k_dev || !v_dev)))
    return fail(AI_ERR_ARG, "null pointer argument");
  if (head_dim != 64 && head_dim != 128) return fail(AI_ERR_ARG, "head_dim must be 64 or 128");
  if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0)
    return fail(AI_ERR_ARG, "query heads must be a multiple of the key heads");
  if (n_heads / n_kv_heads > 128) return fail(AI_ERR_ARG, "more than 128 query heads per key head");
  if (!(scale == scale) || scale - scale != 0.f) return fail(AI_ERR_ARG, "scale must be finite");
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
  a.c2 = scale * kLog2e;
  a.out = static_cast<uint16_t*>(out_dev);
  a.lse = lse_dev;
  a.status = status_dev;
  if (n_seqs > 65535) return fail(AI_ERR_ARG, "more than 65535 sequences");
  const dim3 grid(static_cast<unsigned>(total_q < 4096 ? total_q : 4096), n_seqs);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  count_launch();
  if (head_dim == 64) k_prompt_rows<64><<<grid, 256, 0, st>>>(a);
  else k_prompt_rows<128><<<grid, 256, 0, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? AI_OK : fail(AI_ERR_CUDA, cudaGetErrorString(e));
}
