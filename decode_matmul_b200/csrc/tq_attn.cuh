// tq_attn.cuh -- attention of new tokens over the paged key/value cache.
#pragma once

#include "tq_kv.cuh"

namespace tq {

struct AttnParams {
  KvView c;
  const void* q;  // [m][q_heads][head_dim]
  const int32_t* seq;  // [m] or null
  const int32_t* pos;  // [m]
  void* out;  // [m][q_heads][head_dim]
  int32_t m, q_heads, window;
  float scale;
  int32_t* status;
};

template <int T>
__device__ __forceinline__ float kv_load(const void* p, int64_t i) {
  if constexpr (T == KV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  if constexpr (T == KV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if constexpr (T == KV_E4M3) return float(static_cast<const __nv_fp8_e4m3*>(p)[i]);
  return 0.f;
}

// One warp per row and query head: o = sum_j softmax(scale q.k_j) v_j in one
// pass over the visible keys with the running maximum and sum.
template <int T, bool OUT_BF16>
__global__ void __launch_bounds__(128) attn_kernel(AttnParams p) {
  constexpr int QT = T == KV_BF16 ? KV_BF16 : KV_F16;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (int64_t)p.m * p.q_heads) return;
  const int row = (int)(item / p.q_heads), h = (int)(item % p.q_heads);
  const int D = p.c.head_dim, per = D / 32;
  const int kvh = h / (p.q_heads / p.c.kv_heads);
  const int32_t seq = p.seq ? p.seq[row] : row;
  int32_t pos = p.pos[row];
  if (pos >= 0 && (seq < 0 || seq >= p.c.n_seqs || pos / p.c.page_size >= p.c.max_pages)) {
    if (lane == 0) flag_bad_index(p.status);
    pos = -1;
  }
  const int32_t first = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
  float q[8], o[8];
  for (int i = 0; i < 8; ++i) {
    q[i] = i < per ? kv_load<QT>(p.q, item * D + i * 32 + lane) : 0.f;
    o[i] = 0.f;
  }
  const float ks = p.c.ks ? p.c.ks[kvh] : 1.f, vs = p.c.vs ? p.c.vs[kvh] : 1.f;
  float mx = -INFINITY, sum = 0.f;
  for (int32_t j = first; j <= pos; ++j) {
    const int32_t pi = j / p.c.page_size;
    const int32_t page = p.c.pages[(int64_t)seq * p.c.max_pages + pi];
    if (page < 0 || page >= p.c.n_pages) {
      if (lane == 0) flag_bad_index(p.status);
      continue;
    }
    const int64_t off = (int64_t)page * p.c.page_stride + (int64_t)(j - pi * p.c.page_size) * p.c.token_stride +
                        (int64_t)kvh * p.c.head_stride;
    float s = 0.f;
    for (int i = 0; i < per; ++i) s += q[i] * kv_load<T>(p.c.k, off + i * 32 + lane);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale * ks;
    const float mn = fmaxf(mx, s);
    const float corr = mx == -INFINITY ? 0.f : expf(mx - mn);
    const float e = expf(s - mn);
    sum = sum * corr + e;
    for (int i = 0; i < per; ++i) o[i] = o[i] * corr + e * kv_load<T>(p.c.v, off + i * 32 + lane);
    mx = mn;
  }
  const float inv = sum > 0.f ? vs / sum : (sum == sum ? 0.f : sum);
  for (int i = 0; i < per; ++i) {
    const int64_t at = item * D + i * 32 + lane;
    if constexpr (OUT_BF16)
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o[i] * inv);
    else
      static_cast<__half*>(p.out)[at] = __float2half_rn(o[i] * inv);
  }
}

}  // namespace tq
