// tq_kv.cuh -- the paged key/value cache and the kernel that rotates the
// queries and keys of new tokens and appends keys and values to it.
#pragma once

#include <cuda_fp8.h>

#include "tq_common.cuh"

namespace tq {

// Cache element types (tq.h's TQ_F16, TQ_BF16, TQ_E4M3).
enum { KV_F16 = 1, KV_BF16 = 2, KV_E4M3 = 3 };
constexpr int KV_BAD_INDEX_STATUS = 9;  // TQ_ERR_VALUE

// Device view of a paged cache: element (page, i, head, d) of k and v is at
// page * page_stride + i * token_stride + head * head_stride + d (elements).
struct KvView {
  void* k;
  void* v;
  const int32_t* pages;  // [n_seqs][max_pages]
  const float* ks;       // [kv_heads] or null
  const float* vs;
  int64_t page_stride, token_stride, head_stride;
  int32_t n_pages, page_size, kv_heads, head_dim, n_seqs, max_pages;
};

template <int T>
struct KvElem;
template <>
struct KvElem<KV_F16> {
  using type = __half;
  static constexpr int bytes = 2;
  static __device__ __forceinline__ uint32_t pack2(float a, float b) { return f2_to_h2(a, b); }
};
template <>
struct KvElem<KV_BF16> {
  using type = __nv_bfloat16;
  static constexpr int bytes = 2;
  static __device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
template <>
struct KvElem<KV_E4M3> {
  using type = __nv_fp8_e4m3;
  static constexpr int bytes = 1;
};

__device__ __forceinline__ void flag_bad_index(int32_t* status) { atomicExch(status, KV_BAD_INDEX_STATUS); }

// ---- append --------------------------------------------------------------------
// Per token: q' and k' = the rotated query and key heads, v as it is; q' goes
// to q_out, k' and v to the cache slot of the token's position.
//   pair (a, b) of frequency i: (a cos t - b sin t, a sin t + b cos t),
//   t = pos * freq[i]
// Angles: pos * freq is formed in binary64 in turns (units of 2 pi) and
// reduced to [-1/2, 1/2] there, where binary32 would lose the fraction
// of a turn at far positions (2^17 turns leave 2^-7 of a turn); sine and
// cosine of the reduced angle are binary32.
// 8-bit caches: an e4m3 value is chosen from the binary32 result, except
// where the result is so near to the border between two e4m3 values that its
// rounding errors could decide (about one element in 10^5); those are redone
// in binary64, so that the stored byte is the nearest one to the exact value.
// Bound: memory (the fp32 rows read once, 16- and 8-bit heads written once).
// A thread handles a unit of two runs of 8 features (the two halves of 8 pairs,
// or 16 features in a row), so its loads and 16-bit stores are 16 bytes wide,
// and has its next unit's loads under way.  The block's first threads form the
// token's sines and cosines once for its heads.  Few tokens: the heads of each
// are spread over blocks.  Many: blocks take whole tokens in turn, as many
// blocks as run at once.  Nothing orders the tokens: a slot that two of them
// share gets each of its units from either.
struct AppendParams {
  KvView c;
  const float* qkv;  // [m][qkv_stride]: q heads, k heads, v heads
  int64_t qkv_stride;
  void* q_out;  // [m][q_heads][head_dim]
  const int32_t* seq;  // [m] or null
  const int32_t* pos;  // [m]
  const double* freq;  // [rot / 2]
  int32_t m, q_heads, rot, interleaved;
  int32_t* status;
};

constexpr int AP_THREADS = 128;
// blocks per SM at the kernels' registers
constexpr int append_blocks(int type) { return type == KV_E4M3 ? 5 : 7; }
constexpr double kInvTwoPi = 0.15915494309189533577;

// e4m3 byte nearest to a binary64 value: to binary32 with round-to-odd (the
// last bit records an inexact step, so the second rounding is not misled by a
// false tie), then to e4m3 (ties to even, saturating at 448).
__device__ __forceinline__ uint32_t e4m3_of_double(double d) {
  float f = __double2float_rz(d);
  if ((double)f != d && d == d) f = __uint_as_float(__float_as_uint(f) | 1u);
  return __nv_cvt_float_to_fp8(f, __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// One rotated value in binary64: x cos t + y sin t (y carries the sign).
__device__ __noinline__ uint32_t e4m3_rotated_exact(float x, float y, int32_t pos, double freq, float scale) {
  double t = (double)pos * freq * kInvTwoPi;
  t -= rint(t);
  double s, c;
  sincospi(2.0 * t, &s, &c);
  return e4m3_of_double(((double)x * c + (double)y * s) / (double)scale);
}

__device__ __noinline__ uint32_t e4m3_exact(float x, float scale) { return e4m3_of_double((double)x / (double)scale); }

template <int T>
__device__ __forceinline__ void store_run(void* base, int64_t off, const float v[8]) {
  static_assert(T == KV_F16 || T == KV_BF16, "16-bit store");
  uint4 o;
  o.x = KvElem<T>::pack2(v[0], v[1]);
  o.y = KvElem<T>::pack2(v[2], v[3]);
  o.z = KvElem<T>::pack2(v[4], v[5]);
  o.w = KvElem<T>::pack2(v[6], v[7]);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) = o;
}

template <int T>
__global__ void __launch_bounds__(AP_THREADS, append_blocks(T)) append_kernel(AppendParams p) {
  constexpr int QT = T == KV_BF16 ? KV_BF16 : KV_F16;  // e4m3 caches take fp16 queries
  __shared__ float2 cs[128];
  pdl_wait();
  pdl_launch_dependents();
  const int D = p.c.head_dim;
  const int half = p.rot >> 1;
  const int uph = D >> 4;  // units per head
  const int units = (p.q_heads + 2 * p.c.kv_heads) * uph;
  const int u0 = blockIdx.y * AP_THREADS + threadIdx.x, ustep = gridDim.y * AP_THREADS;
  // the two runs of a unit: features r0 .. r0 + 7 and r1 .. r1 + 7 of its head
  auto runs = [&](int u, int& head, int& w, bool& is_v, bool& turn, bool& halves, int& r0, int& r1) {
    head = u / uph;
    w = u - head * uph;
    is_v = head >= p.q_heads + p.c.kv_heads;
    turn = !is_v && 16 * w < p.rot;
    halves = turn && !p.interleaved;
    r0 = halves ? 8 * w : 16 * w;
    r1 = halves ? half + 8 * w : 16 * w + 8;
  };
  float nx[8], ny[8];  // the next unit, on its way while this one is worked on
  auto load = [&](int t, int u) {
    if (u >= units) {
      t += gridDim.x;
      u = u0;
    }
    if (t >= p.m || u >= units) return;
    int head, w, r0, r1;
    bool is_v, turn, halves;
    runs(u, head, w, is_v, turn, halves, r0, r1);
    const float* row = p.qkv + (int64_t)t * p.qkv_stride + head * D;
    const float4* s0 = reinterpret_cast<const float4*>(row + r0);
    const float4* s1 = reinterpret_cast<const float4*>(row + r1);
    *reinterpret_cast<float4*>(nx) = __ldcs(s0);
    *reinterpret_cast<float4*>(nx + 4) = __ldcs(s0 + 1);
    *reinterpret_cast<float4*>(ny) = __ldcs(s1);
    *reinterpret_cast<float4*>(ny + 4) = __ldcs(s1 + 1);
  };
  load(blockIdx.x, u0);
  int32_t next_pos = p.pos[blockIdx.x];
  for (int t = blockIdx.x; t < p.m; t += gridDim.x) {
    const int32_t pos = next_pos;
    if (t + (int)gridDim.x < p.m) next_pos = p.pos[t + gridDim.x];
    int64_t slot = -1;
    if (pos >= 0) {
      const int32_t seq = p.seq ? p.seq[t] : t;
      const int32_t pi = pos / p.c.page_size;
      int32_t page = -1;
      if (seq >= 0 && seq < p.c.n_seqs && pi < p.c.max_pages) page = p.c.pages[(int64_t)seq * p.c.max_pages + pi];
      if (page >= 0 && page < p.c.n_pages)
        slot = (int64_t)page * p.c.page_stride + (int64_t)(pos - pi * p.c.page_size) * p.c.token_stride;
      else if (threadIdx.x == 0)
        flag_bad_index(p.status);
    }
    __syncthreads();  // the previous token's angles are used
    if (pos >= 0 && (int)threadIdx.x < half) {
      double a = (double)pos * p.freq[threadIdx.x] * kInvTwoPi;
      a -= rint(a);
      float s, c;
      sincospif((float)(2.0 * a), &s, &c);
      cs[threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();
    for (int u = u0; u < units; u += ustep) {
      int head, w, r0, r1;
      bool is_v, turn, halves;
      runs(u, head, w, is_v, turn, halves, r0, r1);
      const bool is_q = head < p.q_heads;
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = nx[i], y[i] = ny[i];
      load(t, u + ustep);
      if (!is_q && slot < 0) continue;
      if (pos < 0) {  // padded row: a zero query
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
      }
      float a[8], b[8];  // results; pairs are (x[i], y[i]) or neighbours inside x and y
      if (!turn || pos < 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = x[i], b[i] = y[i];
      } else if (halves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 r = cs[8 * w + i];
          a[i] = x[i] * r.x - y[i] * r.y;
          b[i] = x[i] * r.y + y[i] * r.x;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 r = cs[8 * w + i], r2 = cs[8 * w + 4 + i];
          a[2 * i] = x[2 * i] * r.x - x[2 * i + 1] * r.y;
          a[2 * i + 1] = x[2 * i] * r.y + x[2 * i + 1] * r.x;
          b[2 * i] = y[2 * i] * r2.x - y[2 * i + 1] * r2.y;
          b[2 * i + 1] = y[2 * i] * r2.y + y[2 * i + 1] * r2.x;
        }
      }
      if (is_q) {
        const int64_t o = ((int64_t)t * p.q_heads + head) * D;
        store_run<QT>(p.q_out, o + r0, a);
        store_run<QT>(p.q_out, o + r1, b);
        continue;
      }
      const int kvh = head - p.q_heads - (is_v ? p.c.kv_heads : 0);
      void* base = is_v ? p.c.v : p.c.k;
      const int64_t o = slot + (int64_t)kvh * p.c.head_stride;
      if constexpr (T != KV_E4M3) {
        store_run<T>(base, o + r0, a);
        store_run<T>(base, o + r1, b);
      } else {
        const float* sp = is_v ? p.c.vs : p.c.ks;
        const float scale = sp ? sp[kvh] : 1.f, inv = 1.f / scale;
        // exact forms only: scales of 0 or NaN, and those whose values or reciprocals may be subnormal (fewer bits)
        const bool odd_scale = !(fabsf(inv) >= 0x1p-100f && fabsf(inv) <= 0x1p100f);
        uint8_t* dst = static_cast<uint8_t*>(base) + o;
#pragma unroll
        for (int run = 0; run < 2; ++run) {
          uint32_t out[2];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            // error of the binary32 value: a few units of the pair's size (the
            // sine, cosine, products, sum, 1 / scale and the product with it each
            // round once: 2^-22 and less of it together)
            const float* val = run ? b : a;
            float e0, e1;
            if (turn) {
              const float n0 = halves ? fabsf(x[i]) + fabsf(y[i]) : (run ? fabsf(y[i]) + fabsf(y[i + 1]) : fabsf(x[i]) + fabsf(x[i + 1]));
              const float n1 = halves ? fabsf(x[i + 1]) + fabsf(y[i + 1]) : n0;
              e0 = n0 * 0x1p-21f;
              e1 = n1 * 0x1p-21f;
            } else {
              e0 = fabsf(val[i]) * 0x1p-22f;
              e1 = fabsf(val[i + 1]) * 0x1p-22f;
            }
            const uint32_t lo = e4m3x2((val[i] - e0) * inv, (val[i + 1] - e1) * inv);
            const uint32_t hi = e4m3x2((val[i] + e0) * inv, (val[i + 1] + e1) * inv);
            uint32_t q2 = hi;
            if (lo != hi || odd_scale) {
              uint32_t b0, b1;
              if (!turn) {
                b0 = e4m3_exact(val[i], scale);
                b1 = e4m3_exact(val[i + 1], scale);
              } else if (halves) {
                const double f0 = p.freq[8 * w + i], f1 = p.freq[8 * w + i + 1];
                b0 = run ? e4m3_rotated_exact(y[i], x[i], pos, f0, scale) : e4m3_rotated_exact(x[i], -y[i], pos, f0, scale);
                b1 = run ? e4m3_rotated_exact(y[i + 1], x[i + 1], pos, f1, scale)
                         : e4m3_rotated_exact(x[i + 1], -y[i + 1], pos, f1, scale);
              } else {
                const float* in = run ? y : x;
                const double f = p.freq[8 * w + 4 * run + (i >> 1)];
                b0 = e4m3_rotated_exact(in[i], -in[i + 1], pos, f, scale);
                b1 = e4m3_rotated_exact(in[i + 1], in[i], pos, f, scale);
              }
              q2 = b0 | (b1 << 8);
            }
            if (i & 2)
              out[i >> 2] |= q2 << 16;
            else
              out[i >> 2] = q2;
          }
          *reinterpret_cast<uint2*>(dst + (run ? r1 : r0)) = make_uint2(out[0], out[1]);
        }
      }
    }
  }
}

}  // namespace tq
