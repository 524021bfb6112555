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

// Step 3 for NT columns of 8 tokens: this warp's groups of 32 features, e0,
// e0 + step, ... below e1.  GN groups are worked on together; B is loaded
// AHEAD steps of 16 ranks at a time, before the steps in hand are multiplied.
// RING: y comes through this warp's two buffers in shared memory, copied a
// round ahead (with 32 tokens its registers would not leave room to have the
// next group's loads in flight).
template <bool BF16, bool VEC, int NT, int GN, int AHEAD, bool RING>
__device__ __forceinline__ void lora_expand(const LoraParams& p, int32_t ad, int e0, int e1, int step, const int32_t* tok,
                                            int cnt, const uint16_t* planes, int pstride, const float* mul, uint8_t* ring) {
  static_assert(!RING || (VEC && GN == 1), "ring");
  constexpr int TERMS = BF16 ? 3 : 2;
  constexpr int STAGE = NT * 8 * 128;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  // MMA rows g, g + 8 of the two row tiles are features 4g .. 4g + 3
  const uint16_t* bp = static_cast<const uint16_t*>(p.b) + (int64_t)ad * p.n * p.rank + q * 4;
  const uint32_t ring_u = RING ? smem_u32(ring) : 0;
  // row c of a stage is token c's 8 chunks of 4 features, chunk i at i ^ ((c >> 1) & 3) * 2
  auto fetch = [&](int e, int stage) {
#pragma unroll
    for (int i = 0; i < NT * 2; ++i) {
      const int c = i * 4 + (lane >> 3), ch = lane & 7, f = e * 32 + ch * 4;
      const bool in = e < e1 && c < cnt && f + 4 <= p.n;
      const float* src = in ? p.y + tok[c] * p.y_stride + f : p.y;
      cp_async16(ring_u + stage * STAGE + c * 128 + (ch ^ (((c >> 1) & 3) * 2)) * 16, src, in);
    }
    cp_async_commit();
  };
  int stage = 0;
  if (RING) fetch(e0, 0);
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
    if (RING) fetch(e + step, stage ^ 1);
    float4 yv[GN][NT][2];
    if (!RING) {
#pragma unroll
      for (int j = 0; j < GN; ++j) {
        const int f = (e + j * step) * 32 + 4 * g;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = nt * 8 + q * 2 + i;
            float4& v = yv[j][nt][i];
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
    }
    float acc[GN][2][NT][4];
#pragma unroll
    for (int j = 0; j < GN; ++j)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[j][mt][nt][i] = 0.f;
    for (int r0 = 0; r0 < p.rank; r0 += 16 * AHEAD) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int r = r0 + u * 16;
        if (r >= p.rank) break;
        uint32_t m0[GN][4], m1[GN][4];
#pragma unroll
        for (int j = 0; j < GN; ++j) {
          m0[j][0] = b[j][u][0].x, m0[j][1] = b[j][u][1].x, m0[j][2] = b[j][u][0].y, m0[j][3] = b[j][u][1].y;
          m1[j][0] = b[j][u][2].x, m1[j][1] = b[j][u][3].x, m1[j][2] = b[j][u][2].y, m1[j][3] = b[j][u][3].y;
        }
#pragma unroll
        for (int term = 0; term < TERMS; ++term)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 h = *reinterpret_cast<const uint2*>(planes + ((term * kLoraTile) + nt * 8 + g) * pstride + r + q * 4);
#pragma unroll
            for (int j = 0; j < GN; ++j) {
              mma16<BF16>(acc[j][0][nt], m0[j], h.x, h.y);
              mma16<BF16>(acc[j][1][nt], m1[j], h.x, h.y);
            }
          }
      }
      if (r0 + 16 * AHEAD < p.rank) load_b(r0 + 16 * AHEAD);
    }
    if (RING) {
      cp_async_wait<1>();
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < GN; ++j) {
      const int f = (e + j * step) * 32 + 4 * g;
      if (e + j * step >= e1) break;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = nt * 8 + q * 2 + i;
          if (c >= cnt || f >= p.n) continue;
          float4 v = yv[j][nt][i];
          if (RING) {
            v = *reinterpret_cast<const float4*>(ring + stage * STAGE + c * 128 + (g ^ (q * 2)) * 16);
            if (f + 4 > p.n) {  // the last features of an odd n were not copied
              const float* src = p.y + tok[c] * p.y_stride + f;
              v.x = src[0];
              if (f + 1 < p.n) v.y = src[1];
              if (f + 2 < p.n) v.z = src[2];
            }
          }
          const float s = mul[c];
          v.x = fmaf(acc[j][0][nt][i], s, v.x);
          v.y = fmaf(acc[j][0][nt][2 + i], s, v.y);
          v.z = fmaf(acc[j][1][nt][i], s, v.z);
          v.w = fmaf(acc[j][1][nt][2 + i], s, v.w);
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
    stage ^= 1;
    if (RING) __syncwarp();  // the buffer is read before it is filled again
  }
}

// Shared memory of a block.  The copies of y (step 3) take the place of the
// sums of A x (steps 1 and 2).
struct LoraSmem {
  static constexpr int PSTRIDE = 128 + 16;  // a token's terms, 8 words past a multiple of 32 (no bank conflicts)
  static constexpr int WARPS = LORA_THREADS / 32;
  int32_t ids[kLoraInBlock], tok[kLoraTile], head[4], lead_count[WARPS];
  float mul[kLoraTile];
  uint16_t planes[3 * kLoraTile * PSTRIDE];  // [term][token][rank]
  union alignas(16) {
    struct {
      float h[128 * kLoraTile];      // the block's sum: [rank][token]
      float total[128 * kLoraTile];  // the cluster's
      float warp[WARPS * 16 * kLoraTile];
    };
    uint8_t ring[WARPS * 2 * kLoraTile * 128];
  };
};

template <bool BF16, bool VEC>
__global__ void __cluster_dims__(LORA_CLUSTER, 1, 1) __launch_bounds__(LORA_THREADS, 2)
    lora_kernel(const __grid_constant__ LoraParams p) {
  constexpr int WARPS = LORA_THREADS / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  LoraSmem& sm = *reinterpret_cast<LoraSmem*>(smem);
  int32_t *ids = sm.ids, *tok = sm.tok, *head = sm.head, *lead_count = sm.lead_count;

  cg::cluster_group cluster = cg::this_cluster();
  const int part = cluster.block_rank();
  const int tile = blockIdx.x / LORA_CLUSTER;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();
  pdl_launch_dependents();

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
  for (int c = warp; c < cols; c += WARPS) {
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
        sm.planes[(term * kLoraTile + c) * LoraSmem::PSTRIDE + r] = t;
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
  const int groups = (p.n + 31) >> 5;
  const int e0 = (int)((int64_t)groups * part / LORA_CLUSTER) + warp, e1 = (int)((int64_t)groups * (part + 1) / LORA_CLUSTER);
  uint8_t* ring = sm.ring + warp * 2 * kLoraTile * 128;
  if (cnt <= 8)
    lora_expand<BF16, VEC, 1, 2, 2, false>(p, ad, e0, e1, WARPS, tok, cnt, sm.planes, LoraSmem::PSTRIDE, sm.mul, ring);
  else if (cnt <= 16)
    lora_expand<BF16, VEC, 2, 1, 4, VEC>(p, ad, e0, e1, WARPS, tok, cnt, sm.planes, LoraSmem::PSTRIDE, sm.mul, ring);
  else
    lora_expand<BF16, VEC, 4, 1, 4, VEC>(p, ad, e0, e1, WARPS, tok, cnt, sm.planes, LoraSmem::PSTRIDE, sm.mul, ring);
  if (VEC) cp_async_wait<0>();
}

}  // namespace tq
