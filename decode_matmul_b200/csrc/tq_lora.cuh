// tq_lora.cuh -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = y[t] + s_a B_a (A_a x_t),   a = the token's adapter
//
// Bound: memory.  The adapters that are used, x and y are read once and out is
// written once; the products are a few per cent of the tensor rate.
// Tokens of one adapter are worked on together, up to 32 in a tile (stable
// order), by one cluster of eight blocks:
//   1. h = A x: the cluster's warps split k (and the 16-row tiles of A); each
//      reads its pieces of A and x straight into MMA fragments (16-byte loads;
//      the order of k inside an MMA is permuted alike for both),
//   2. the blocks' sums of h are exchanged through distributed shared memory,
//      so no second launch and no trip through global memory is needed,
//   3. each block takes an eighth of the n output features: B as the 16-row
//      operand, tokens as the 8-wide one, 32 features in an order that gives a
//      thread four neighbours (16-byte accesses of y and out).
// A x keeps binary32 accuracy through the second product: it enters as three
// bf16 terms (24 bits), or as two fp16 terms of a token's h scaled by a power
// of two (22 bits of its largest element).
#pragma once

#include <cooperative_groups.h>

#include "tq_attn.cuh"
#include "tq_umma.cuh"

namespace tq {

namespace cg = cooperative_groups;

struct LoraParams {
  const void* a;       // [n_adapters][rank][k]
  const void* b;       // [n_adapters][n][rank]
  const float* scale;  // [n_adapters] or null
  const void* x;       // [m][k]
  const int32_t* adapter;  // [m]
  const float* y;      // rows of y_stride
  float* out;          // rows of out_stride
  int64_t y_stride, out_stride;
  int32_t n_adapters, rank, n, k, m;
  int32_t* plan;  // workspace (m > kLoraInBlock): tiles, perm [4096], first [4097]
  int32_t* status;
};

// 16 consecutive 32-bit TMEM columns of this thread's lane (warp-collective)
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

constexpr int LORA_THREADS = 256;
constexpr int LORA_CLUSTER = 8;
constexpr int kLoraTile = 32;      // tokens of a tile
constexpr int kLoraInBlock = 256;  // up to this many tokens each block groups them for itself
constexpr int kLoraMaxM = 4096;
constexpr int kPlanPerm = 4, kPlanFirst = kPlanPerm + kLoraMaxM, kPlanInts = kPlanFirst + kLoraMaxM + 4;

__device__ __forceinline__ int32_t lora_adapter(const LoraParams& p, int t, bool& bad) {
  const int32_t a = p.adapter[t];
  bad = a >= p.n_adapters;
  return a < 0 || bad ? -1 : a;
}

// Grouping of more than kLoraInBlock tokens, by one block: a stable radix sort
// of (adapter, token) in shared memory, five bits a pass (40 adapters: two
// passes), then a list of where each tile begins in the sorted order.  A warp
// takes 128 tokens in their order, 32 at a time; lanes with the same digit find
// one another by a match, so no atomics are needed and the order is always the
// same.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const __grid_constant__ LoraParams p) {
  __shared__ uint32_t key[2][kLoraMaxM];  // (adapter + 1) << 12 | token
  __shared__ int32_t count[32][33];  // [digit][warp]
  __shared__ int32_t warp_sum[32], warp_max[32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = i * 1024 + tid;
    uint32_t v = 0xffffffffu;  // behind the last token
    if (t < p.m) {
      bool bad;
      v = (uint32_t)(lora_adapter(p, t, bad) + 1) << 12 | (uint32_t)t;
      if (bad) flag_bad_index(p.status);
    }
    key[0][t] = v;
  }
  int cur = 0;
  const int bits = 32 - __clz(p.n_adapters + 1);  // so that the padding's bits are above all adapters'
  for (int shift = 12; shift < 12 + bits; shift += 5) {
    count[lane][warp] = 0;
    __syncthreads();
    uint32_t v[4];
    int32_t rank[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = warp * 128 + i * 32 + lane;
      v[i] = key[cur][at];
      const int digit = (v[i] >> shift) & 31;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      const int first = __ffs(same) - 1;
      const int base = count[digit][warp];
      __syncwarp();
      if (lane == first) count[digit][warp] = base + __popc(same);
      __syncwarp();
      rank[i] = base + __popc(same & ((1u << lane) - 1));
    }
    __syncthreads();
    // exclusive sums over (digit, warp) in that order: thread (d = warp, w = lane)
    const int32_t c = count[warp][lane];
    int32_t incl = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t u = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += u;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int32_t prior = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) prior += __shfl_xor_sync(0xffffffffu, prior, d);
    count[warp][lane] = prior + incl - c;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int to = count[(v[i] >> shift) & 31][warp] + rank[i];
      key[cur ^ 1][to] = v[i];
    }
    cur ^= 1;
    __syncthreads();
  }
  // a thread has four neighbours; a group's tiles begin every kLoraTile tokens of it
  const int i0 = tid * 4;
  int32_t start[4];  // where the token's group begins
  int32_t run = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i0 + i;
    if (at < p.m && (at == 0 || (key[cur][at] >> 12) != (key[cur][at - 1] >> 12))) run = at;
    start[i] = run;
  }
  int32_t before = run;  // inclusive running maximum over threads
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t v = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before = max(before, v);
  }
  if (lane == 31) warp_max[warp] = before;
  __syncthreads();
  int32_t prev = __shfl_up_sync(0xffffffffu, before, 1);
  if (lane == 0) prev = -1;
  for (int w = 0; w < warp; ++w) prev = max(prev, warp_max[w]);
  int32_t lead = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    start[i] = max(start[i], prev);
    const int at = i0 + i;
    if (at < p.m) {
      p.plan[kPlanPerm + at] = (int32_t)(key[cur][at] & 4095u);
      if ((at - start[i]) % kLoraTile == 0) ++lead;
    }
  }
  int32_t incl = lead;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int32_t at_tile = incl - lead, total = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) at_tile += warp_sum[w];
    total += warp_sum[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i0 + i;
    if (at < p.m && (at - start[i]) % kLoraTile == 0) p.plan[kPlanFirst + at_tile++] = at;
  }
  if (tid == 0) {
    p.plan[0] = total;
    p.plan[kPlanFirst + total] = p.m;
  }
}

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Step 1 for NT columns of 8 tokens: this warp's sum over its k pieces.
template <bool BF16, int NT>
__device__ __forceinline__ void lora_shrink(const LoraParams& p, int32_t ad, int rt, const int32_t* tok, int cnt, int g0,
                                            int g1, float* hp) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int r0 = rt * 16 + g, r1 = r0 + 8;
  const uint16_t* a0 = static_cast<const uint16_t*>(p.a) + ((int64_t)ad * p.rank + r0) * p.k + q * 8;
  const uint16_t* a1 = a0 + (r1 < p.rank ? (int64_t)8 * p.k : 0);
  const bool two = r1 < p.rank;
  const uint16_t* xp[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = nt * 8 + g;
    xp[nt] = static_cast<const uint16_t*>(p.x) + (int64_t)tok[c < cnt ? c : 0] * p.k + q * 8;
  }
  float acc[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
  constexpr int U = NT == 4 ? 3 : (NT == 2 ? 4 : 8);  // pieces of 32 features in flight together
  for (int gi = g0; gi < g1; gi += U) {
    uint4 a[U][2], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = (int64_t)(gi + u < g1 ? gi + u : g1 - 1) * 32;
      a[u][0] = ldg16(a0 + o);
      a[u][1] = ldg16(a1 + o);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[u][nt] = ldg16(xp[nt] + o);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (gi + u >= g1) break;
      if (!two) a[u][1] = make_uint4(0, 0, 0, 0);
      const uint32_t f0[4] = {a[u][0].x, a[u][1].x, a[u][0].y, a[u][1].y};
      const uint32_t f1[4] = {a[u][0].z, a[u][1].z, a[u][0].w, a[u][1].w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma16<BF16>(acc[nt], f0, x[u][nt].x, x[u][nt].y);
        mma16<BF16>(acc[nt], f1, x[u][nt].z, x[u][nt].w);
      }
    }
  }
  // [rank in tile][token]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    *reinterpret_cast<float2*>(hp + g * kLoraTile + nt * 8 + q * 2) = make_float2(acc[nt][0], acc[nt][1]);
    *reinterpret_cast<float2*>(hp + (g + 8) * kLoraTile + nt * 8 + q * 2) = make_float2(acc[nt][2], acc[nt][3]);
  }
}

// Step 3 for up to 8 tokens: this warp's groups of 32 features, e0, e0 + step,
// ... below e1, two at a time with all their loads in flight (B 32 ranks at a
// time, the next while these are multiplied).
template <bool BF16, bool VEC>
__device__ __forceinline__ void lora_expand8(const LoraParams& p, int32_t ad, int e0, int e1, int step, const int32_t* tok,
                                             int cnt, const uint16_t* planes, int pstride, const float* mul) {
  constexpr int GN = 2, AHEAD = 2;
  constexpr int TERMS = BF16 ? 3 : 2;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  // MMA rows g, g + 8 of the two row tiles are features 4g .. 4g + 3
  const uint16_t* bp = static_cast<const uint16_t*>(p.b) + (int64_t)ad * p.n * p.rank + q * 4;
  for (int e = e0; e < e1; e += GN * step) {
    uint2 b[GN][AHEAD][4];
    auto load_b = [&](int r0) {
#pragma unroll
      for (int j = 0; j < GN; ++j) {
        const int f = (e + j * step) * 32 + 4 * g;
        const bool on = e + j * step < e1;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int r = r0 + u * 16;
          const bool in = on && r + q * 4 < p.rank;  // false too in the last 8 of an odd number of eights
#pragma unroll
          for (int i = 0; i < 4; ++i)
            b[j][u][i] = in && f + i < p.n ? __ldg(reinterpret_cast<const uint2*>(bp + (int64_t)(f + i) * p.rank + r))
                                           : make_uint2(0, 0);
        }
      }
    };
    load_b(0);
    float4 yv[GN][2];
#pragma unroll
    for (int j = 0; j < GN; ++j) {
      const int f = (e + j * step) * 32 + 4 * g;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = q * 2 + i;
        float4& v = yv[j][i];
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e + j * step < e1 && c < cnt && f < p.n) {
          const float* src = p.y + tok[c] * p.y_stride + f;
          if (VEC && f + 4 <= p.n) {
            v = *reinterpret_cast<const float4*>(src);
          } else {
            v.x = src[0];
            if (f + 1 < p.n) v.y = src[1];
            if (f + 2 < p.n) v.z = src[2];
            if (f + 3 < p.n) v.w = src[3];
          }
        }
      }
    }
    float acc[GN][2][4];
#pragma unroll
    for (int j = 0; j < GN; ++j)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][mt][i] = 0.f;
    for (int r0 = 0; r0 < p.rank; r0 += 16 * AHEAD) {
      uint2 now[GN][AHEAD][4];
#pragma unroll
      for (int j = 0; j < GN; ++j)
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) now[j][u][i] = b[j][u][i];
      if (r0 + 16 * AHEAD < p.rank) load_b(r0 + 16 * AHEAD);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int r = r0 + u * 16;
        if (r >= p.rank) break;
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          const uint2 h = *reinterpret_cast<const uint2*>(planes + (term * 8 + g) * pstride + r + q * 4);
#pragma unroll
          for (int j = 0; j < GN; ++j) {
            const uint32_t m0[4] = {now[j][u][0].x, now[j][u][1].x, now[j][u][0].y, now[j][u][1].y};
            const uint32_t m1[4] = {now[j][u][2].x, now[j][u][3].x, now[j][u][2].y, now[j][u][3].y};
            mma16<BF16>(acc[j][0], m0, h.x, h.y);
            mma16<BF16>(acc[j][1], m1, h.x, h.y);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < GN; ++j) {
      const int f = (e + j * step) * 32 + 4 * g;
      if (e + j * step >= e1) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = q * 2 + i;
        if (c >= cnt || f >= p.n) continue;
        const float s = mul[c];
        float4 v = yv[j][i];
        v.x = fmaf(acc[j][0][i], s, v.x);
        v.y = fmaf(acc[j][0][2 + i], s, v.y);
        v.z = fmaf(acc[j][1][i], s, v.z);
        v.w = fmaf(acc[j][1][2 + i], s, v.w);
        float* dst = p.out + tok[c] * p.out_stride + f;
        if (VEC && f + 4 <= p.n) {
          *reinterpret_cast<float4*>(dst) = v;
        } else {
          dst[0] = v.x;
          if (f + 1 < p.n) dst[1] = v.y;
          if (f + 2 < p.n) dst[2] = v.z;
          if (f + 3 < p.n) dst[3] = v.w;
        }
      }
    }
  }
}

// Shared memory of a block.  In step 3 the tiles of B (9 to 32 tokens) take
// the place of the sums of A x (steps 1 and 2).
struct LoraSmem {
  static constexpr int PSTRIDE = 128 + 16;  // a token's terms, 8 words past a multiple of 32 (no bank conflicts)
  static constexpr int WARPS = LORA_THREADS / 32;
  static constexpr int PANEL_B = 128 * 128;         // 128 features x 64 ranks
  static constexpr int PANEL_H = kLoraTile * 128;   // 32 tokens x 64 ranks
  union {
    struct {
      float h[128 * kLoraTile];      // the block's sum: [rank][token]
      float total[128 * kLoraTile];  // the cluster's
      float warp[WARPS * 16 * kLoraTile];
    };
    uint8_t b[2][2 * PANEL_B];  // two tiles of 128 features, up to 128 ranks
  };
  union {
    uint16_t planes[3 * 8 * PSTRIDE];  // up to 8 tokens: [term][token][rank]
    uint8_t terms[3][2 * PANEL_H];     // more: operand tiles
  };
  int64_t yoff[kLoraTile], ooff[kLoraTile];  // the tokens' rows of y and out
  uint64_t bar[2];
  int32_t ids[kLoraInBlock], tok[kLoraTile], head[4], lead_count[WARPS];
  float mul[kLoraTile];
  uint32_t tmem;
};

// Step 3 for 9 to 32 tokens, on the tcgen05 tensor cores: D [128 features][32
// tokens] = B [128][rank] (terms of h)^T.  Read out of shared memory by the
// tensor core, the operands cost the threads nothing: with warp MMAs their
// fragments (and the addresses of 8 tokens' y per thread) took 1350
// instructions per 32 x 32 outputs and 54 us of 1000 tokens x 19456 features
// at rank 64.  The next tile of B is copied and its y loaded while this one is
// multiplied; each thread has one feature and 16 tokens, so a warp's accesses
// of y and out are 128 bytes in a row at any alignment.
template <bool BF16>
__device__ __forceinline__ void lora_expand32(const LoraParams& p, int32_t ad, int cnt, int part, LoraSmem& sm) {
  constexpr int TERMS = BF16 ? 3 : 2;
  constexpr uint32_t IDESC = (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | ((kLoraTile >> 3) << 17) | ((128 >> 4) << 24);
  constexpr int COLS = kLoraTile / 2;  // tokens of a thread
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int panels = (p.rank + 63) >> 6, steps = (p.rank + 15) >> 4;
  const int tiles = (p.n + 127) >> 7;
  const int t0 = tiles * part / LORA_CLUSTER, t1 = tiles * (part + 1) / LORA_CLUSTER;
  const uint32_t bar = smem_u32(sm.bar), tmem = sm.tmem;
  const uint16_t* bsrc = static_cast<const uint16_t*>(p.b) + (int64_t)ad * p.n * p.rank;
  // rows of 64 ranks are 128 bytes, 16-byte chunk i of row r at i ^ (r & 7)
  // (the 128-byte swizzle); ranks up to the last step of 16 that are not there
  // are zeros
  auto fetch = [&](int t) {
    const uint32_t dst = smem_u32(sm.b[t & 1]);
    for (int pn = 0; pn < panels; ++pn) {
      const int chunks = min(8, steps * 2 - pn * 8);
      const int ch = tid & 7;
      if (ch < chunks) {
        const int r = pn * 64 + ch * 8;
#pragma unroll
        for (int i = 0; i < 128 * 8 / LORA_THREADS; ++i) {
          const int row = i * (LORA_THREADS / 8) + (tid >> 3), f = t * 128 + row;
          const bool in = f < p.n && r < p.rank;
          cp_async16(dst + pn * LoraSmem::PANEL_B + row * 128 + ((ch ^ (row & 7)) << 4),
                     in ? bsrc + (int64_t)f * p.rank + r : bsrc, in);
        }
      }
    }
  };
  const int c0 = (warp >> 2) * COLS;
  const int row = (warp & 3) * 32 + lane;
  float yv[COLS];
  auto load_y = [&](int t) {
    const int f = t * 128 + row;
#pragma unroll
    for (int j = 0; j < COLS; ++j) yv[j] = c0 + j < cnt && f < p.n && t < t1 ? p.y[sm.yoff[c0 + j] + f] : 0.f;
  };
  if (t0 < t1) fetch(t0);
  cp_async_commit();
  load_y(t0);
  bool good = true;
  for (int t = t0; t < t1; ++t) {
    if (t + 1 < t1) fetch(t + 1);  // into the buffer whose products the previous round waited for
    cp_async_commit();
    cp_async_wait<1>();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    const int it = t - t0;
    const uint32_t d = tmem + (it & 1) * kLoraTile;
    if (tid == 0) {
      tc_fence_after();
      for (int k = 0; k < steps; ++k) {
        const uint64_t a = umma_smem_desc(smem_u32(sm.b[t & 1]) + (k >> 2) * LoraSmem::PANEL_B + (k & 3) * 32);
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
          umma_f16(d, a, umma_smem_desc(smem_u32(sm.terms[term]) + (k >> 2) * LoraSmem::PANEL_H + (k & 3) * 32), IDESC,
                   k + term > 0);
      }
      umma_commit(bar + 8 * (it & 1));
    }
    float v[COLS];
#pragma unroll
    for (int j = 0; j < COLS; ++j) v[j] = yv[j];
    load_y(t + 1);
    // a wait that runs out (it cannot in a healthy launch) leaves the outputs undefined and says so
    good = __all_sync(0xffffffffu, mbar_wait(bar + 8 * (it & 1), (it >> 1) & 1, 1u << 21));
    if (!good) {
      if (lane == 0) atomicExch(p.status, UM_TIMEOUT_STATUS);
      continue;
    }
    tc_fence_after();
    uint32_t acc[COLS];
    tmem_ld16(d + ((uint32_t)((warp & 3) * 32) << 16) + c0, acc);
    const int f = t * 128 + row;
#pragma unroll
    for (int j = 0; j < COLS; ++j)
      if (c0 + j < cnt && f < p.n) p.out[sm.ooff[c0 + j] + f] = fmaf(__uint_as_float(acc[j]), sm.mul[c0 + j], v[j]);
  }
  cp_async_wait<0>();
}

template <bool BF16, bool VEC>
__global__ void __cluster_dims__(LORA_CLUSTER, 1, 1) __launch_bounds__(LORA_THREADS, 2)
    lora_kernel(const __grid_constant__ LoraParams p) {
  constexpr int WARPS = LORA_THREADS / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  LoraSmem& sm = *reinterpret_cast<LoraSmem*>(smem + (-smem_u32(smem) & 1023u));  // the operand tiles are aligned to 1 KB
  int32_t *ids = sm.ids, *tok = sm.tok, *head = sm.head, *lead_count = sm.lead_count;

  cg::cluster_group cluster = cg::this_cluster();
  const int part = cluster.block_rank();
  const int tile = blockIdx.x / LORA_CLUSTER;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();

  // ---- the tile's tokens -------------------------------------------------------
  int cnt;
  int32_t ad;
  if (p.m > kLoraInBlock) {
    if (tile >= p.plan[0]) return;  // the whole cluster
    const int i0 = p.plan[kPlanFirst + tile];
    cnt = p.plan[kPlanFirst + tile + 1] - i0;
    if (tid < cnt) tok[tid] = p.plan[kPlanPerm + i0 + tid];
    bool bad;
    ad = lora_adapter(p, p.plan[kPlanPerm + i0], bad);
    __syncthreads();
  } else {
    int32_t id = -1;
    if (tid < p.m) {
      bool bad;
      id = lora_adapter(p, tid, bad);
      if (bad && blockIdx.x == 0) flag_bad_index(p.status);
    }
    ids[tid] = id;
    if (tid == 0) head[0] = -1;
    __syncthreads();
    // how many tokens of the same adapter come before this one
    int before = 0;
    if (tid < p.m) {
      const int4* v = reinterpret_cast<const int4*>(ids);
      for (int s = 0; s < tid; s += 4) {
        const int4 o = v[s >> 2];
        before += (o.x == id) + (s + 1 < tid && o.y == id) + (s + 2 < tid && o.z == id) + (s + 3 < tid && o.w == id);
      }
    }
    const bool lead = tid < p.m && before % kLoraTile == 0;
    const uint32_t leads = __ballot_sync(0xffffffffu, lead);
    if (lane == 0) lead_count[warp] = __popc(leads);
    __syncthreads();
    int mine = __popc(leads & ((1u << lane) - 1)), total = 0;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) mine += lead_count[w];
      total += lead_count[w];
    }
    if (tile >= total) return;  // the whole cluster
    if (lead && mine == tile) {
      head[0] = id;
      head[1] = before;
      head[2] = 0;
    }
    __syncthreads();
    ad = head[0];
    const int first = head[1];
    const bool in = tid < p.m && id == ad && before >= first && before < first + kLoraTile;
    if (in) tok[before - first] = tid;
    cnt = __syncthreads_count(in);
  }

  if (ad < 0) {  // no adapter: y as it is
    if (warp == 0) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    if (p.out != p.y)
      for (int c = 0; c < cnt; ++c) {
        const float* src = p.y + tok[c] * p.y_stride;
        float* dst = p.out + tok[c] * p.out_stride;
        if (VEC) {
          const int quads = p.n >> 2;
          for (int i = part * LORA_THREADS + tid; i < quads; i += LORA_CLUSTER * LORA_THREADS)
            reinterpret_cast<float4*>(dst)[i] = reinterpret_cast<const float4*>(src)[i];
          for (int i = quads * 4 + part * LORA_THREADS + tid; i < p.n; i += LORA_CLUSTER * LORA_THREADS) dst[i] = src[i];
        } else {
          for (int i = part * LORA_THREADS + tid; i < p.n; i += LORA_CLUSTER * LORA_THREADS) dst[i] = src[i];
        }
      }
    return;
  }

  const bool wide = cnt > 8;  // step 3 on the tcgen05 tensor cores
  // every block gives up its right to allocate tensor memory at once: until it
  // does, no second block of this kernel starts on its SM (64 tokens of 24
  // adapters: 34 us with one block per SM at a time, 20 us with two)
  if (!wide && warp == 0) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  if (wide) {
    if (warp == 0) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sm.tmem)), "r"(64u));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (tid == 32) {
      mbar_init(smem_u32(sm.bar), 1);
      mbar_init(smem_u32(sm.bar) + 8, 1);
      asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid >= 64 && tid < 64 + cnt) {
      sm.yoff[tid - 64] = tok[tid - 64] * p.y_stride;
      sm.ooff[tid - 64] = tok[tid - 64] * p.out_stride;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  // only now: the next kernel may take tensor memory before it waits for this one
  pdl_launch_dependents();

  // ---- 1. h = A x over this block's share of k -----------------------------------
  const int rts = (p.rank + 15) >> 4;         // 16-row tiles of A
  const int kparts = WARPS / rts;             // warps that share a tile's k
  const int rt = warp / kparts, kp = warp - rt * kparts;
  if (rt < rts) {
    const int pieces = p.k >> 5, shares = LORA_CLUSTER * kparts, s = part * kparts + kp;
    const int g0 = (int)((int64_t)pieces * s / shares), g1 = (int)((int64_t)pieces * (s + 1) / shares);
    float* to = sm.warp + warp * 16 * kLoraTile;
    if (cnt <= 8)
      lora_shrink<BF16, 1>(p, ad, rt, tok, cnt, g0, g1, to);
    else if (cnt <= 16)
      lora_shrink<BF16, 2>(p, ad, rt, tok, cnt, g0, g1, to);
    else
      lora_shrink<BF16, 4>(p, ad, rt, tok, cnt, g0, g1, to);
  }
  __syncthreads();
  const int cols = cnt <= 8 ? 8 : (cnt <= 16 ? 16 : 32), cshift = cnt <= 8 ? 3 : (cnt <= 16 ? 4 : 5);
  const int entries = p.rank << cshift;
  for (int i = tid; i < entries; i += LORA_THREADS) {
    const int r = i >> cshift, c = i & (cols - 1);
    const float* src = sm.warp + (r >> 4) * kparts * 16 * kLoraTile + (r & 15) * kLoraTile + c;
    float s = 0.f;
    for (int w = 0; w < kparts; ++w) s += src[w * 16 * kLoraTile];
    sm.h[i] = s;
  }
  cluster.sync();

  // ---- 2. the cluster's sum, as terms of the operand type --------------------------
  // few entries: every block adds up all of them; more: each adds up an eighth
  // and sends it to all
  {
    const bool all = entries <= 512;
    const int quads = entries >> 2, i0 = all ? 0 : quads * part / LORA_CLUSTER;
    const int i1 = all ? quads : quads * (part + 1) / LORA_CLUSTER;
    for (int i = i0 + tid; i < i1; i += LORA_THREADS) {
      float4 v[LORA_CLUSTER];
#pragma unroll
      for (int b = 0; b < LORA_CLUSTER; ++b) v[b] = reinterpret_cast<const float4*>(cluster.map_shared_rank(sm.h, b))[i];
#pragma unroll
      for (int b = 1; b < LORA_CLUSTER; ++b) v[0].x += v[b].x, v[0].y += v[b].y, v[0].z += v[b].z, v[0].w += v[b].w;
      if (all) {
        reinterpret_cast<float4*>(sm.total)[i] = v[0];
      } else {
#pragma unroll
        for (int b = 0; b < LORA_CLUSTER; ++b) reinterpret_cast<float4*>(cluster.map_shared_rank(sm.total, b))[i] = v[0];
      }
    }
    if (all)
      __syncthreads();
    else
      cluster.sync();
  }
  // one warp per token: lane l has ranks l, l + 32, ...
  const float sa = p.scale ? p.scale[ad] : 1.f;
  const int ranks = rts * 16;  // the last tile's missing ranks are zero terms
  // (with more than 8 tokens the operand tile's 32 rows, all of them)
  for (int c = warp; c < (wide ? kLoraTile : 8); c += WARPS) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = j * 32 + lane;
      v[j] = r < p.rank && c < cnt ? sm.total[(r << cshift) + c] : 0.f;
    }
    float up = 1.f;  // what the scaled terms are multiplied by
    if constexpr (!BF16) {
      float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      // the largest element goes to [2^9, 2^10)
      const int e = (int)((__float_as_uint(top) >> 23) & 255) - 127;
      if (e > -110 && e < 120) {
        up = __uint_as_float((uint32_t)(e - 9 + 127) << 23);
        const float down = __uint_as_float((uint32_t)(9 - e + 127) << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= down;
      }
    }
    if (lane == 0) sm.mul[c] = sa * up;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = j * 32 + lane;
      if (r >= ranks) continue;
      float rest = v[j];
#pragma unroll
      for (int term = 0; term < (BF16 ? 3 : 2); ++term) {
        const uint16_t t = BF16 ? f_to_bf16_bits(rest) : __half_as_ushort(__float2half_rn(rest));
        if (!wide)
          sm.planes[(term * 8 + c) * LoraSmem::PSTRIDE + r] = t;
        else
          *reinterpret_cast<uint16_t*>(sm.terms[term] + (r >> 6) * LoraSmem::PANEL_H + c * 128 +
                                       ((((r >> 3) & 7) ^ (c & 7)) << 4) + (r & 7) * 2) = t;
        const float back = BF16 ? bf16_bits_to_f(t) : __half2float(__ushort_as_half(t));
        rest = fabsf(back) < INFINITY ? rest - back : 0.f;
      }
    }
  }
  // before copies of y take the place of the sums, and before a block leaves,
  // the others have read its h (those who got the sums sent have already)
  if (entries <= 512)
    cluster.sync();
  else
    __syncthreads();

  // ---- 3. out = y + s B h over this block's share of n -------------------------------
  if (!wide) {
    const int groups = (p.n + 31) >> 5;
    const int e0 = (int)((int64_t)groups * part / LORA_CLUSTER) + warp;
    const int e1 = (int)((int64_t)groups * (part + 1) / LORA_CLUSTER);
    lora_expand8<BF16, VEC>(p, ad, e0, e1, WARPS, tok, cnt, sm.planes, LoraSmem::PSTRIDE, sm.mul);
    return;
  }
  lora_expand32<BF16>(p, ad, cnt, part, sm);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(sm.tmem), "r"(64u));
  }
}

}  // namespace tq
