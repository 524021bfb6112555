// tq_lora.cuh -- low-rank adapters of many requests beside a shared projection.
#pragma once

#include "tq_kv.cuh"

namespace tq {

struct LoraParams {
  const void* a;       // [n_adapters][rank][k]
  const void* b;       // [n_adapters][n][rank]
  const float* scale;  // [n_adapters] or null
  const void* x;       // [m][k]
  const int32_t* adapter;  // [m]
  const float* y;      // [m][y_stride]
  float* out;          // [m][out_stride]
  int64_t y_stride, out_stride;
  int32_t n_adapters, rank, n, k, m;
  float* h;  // workspace: [m][rank]
  int32_t* status;
};

template <bool BF16>
__device__ __forceinline__ float ld16(const void* p, int64_t i) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

// h = A x: one block per token, one warp per rank at a time.
template <bool BF16>
__global__ void __launch_bounds__(256) lora_shrink_kernel(LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int32_t ad = p.adapter[t];
  if (ad < 0) return;
  if (ad >= p.n_adapters) {
    if (threadIdx.x == 0) flag_bad_index(p.status);
    return;
  }
  for (int r = threadIdx.x >> 5; r < p.rank; r += 8) {
    const int64_t arow = ((int64_t)ad * p.rank + r) * p.k;
    float s = 0.f;
    for (int i = lane; i < p.k; i += 32) s += ld16<BF16>(p.a, arow + i) * ld16<BF16>(p.x, (int64_t)t * p.k + i);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) p.h[(int64_t)t * p.rank + r] = s;
  }
}

// y' = y + s B h: a thread per output feature.
template <bool BF16>
__global__ void __launch_bounds__(256) lora_expand_kernel(LoraParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x;
  const int n = blockIdx.y * 256 + threadIdx.x;
  if (n >= p.n) return;
  const int32_t ad = p.adapter[t];
  float v = p.y[(int64_t)t * p.y_stride + n];
  if (ad >= 0 && ad < p.n_adapters) {
    float s = 0.f;
    for (int r = 0; r < p.rank; ++r)
      s += ld16<BF16>(p.b, ((int64_t)ad * p.n + n) * p.rank + r) * p.h[(int64_t)t * p.rank + r];
    v += (p.scale ? p.scale[ad] : 1.f) * s;
  }
  p.out[(int64_t)t * p.out_stride + n] = v;
}

}  // namespace tq
