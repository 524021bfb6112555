// tq_lora.cuh -- low-rank adapters of many requests beside a shared projection.
//
//   out[t] = y[t] + s_a B_a (A_a x_t),   a = the token's adapter
//
// Bound: memory.  The adapters that are used, x and y are read once and out is
// written once; the products are a few per cent of the tensor rate.  Tokens of
// one adapter are worked on together, so that its A and B are read once for
// all of them.
//
// Up to 256 tokens (decoding), one launch: tiles of up to 8 tokens, each by a
// cluster of eight blocks:
//   1. h = A x: the cluster's warps split k (and the 16-row tiles of A); each
//      reads its pieces of A and x straight into MMA fragments (16-byte loads;
//      the order of k inside an MMA is permuted alike for both),
//   2. the blocks' sums of h are read through distributed shared memory: no
//      second launch, no trip through global memory,
//   3. each block takes an eighth of the n output features: B as the 16-row
//      operand, tokens as the 8-wide one, 32 features in an order that gives a
//      thread four neighbours (16-byte accesses of y and out).
// More tokens (prompts), three launches: the tokens are grouped, h is summed
// over splits of k into the workspace, and tiles of 128 features x 32 tokens
// are multiplied on the tcgen05 tensor cores, whose operands cost the threads
// nothing (with warp MMAs the fragments and addresses took 1350 instructions
// per 32 x 32 outputs).
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
  // workspace, m > kLoraInBlock
  int32_t* plan;    // tiles, perm [4096], of each tile (first in perm, tokens, adapter or -1, 0) [4096]
  float* h;         // of each split, in perm's order: A x of each tile as [rank][its tokens]
  uint16_t* terms;  // in perm's order: [m][3][rank], A x as terms of the operand type
  float* mul;       // in perm's order: what the token's sums are multiplied by
  int32_t splits;   // of k
  int32_t* counters;
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
// Up to this many tokens each block groups them for itself (a thread per token)
// and the call is one launch.  One against three launches, n = 4096, k = 14336,
// rank 16: 64 tokens of 40 adapters 12.8 against 28.2 us, 256 of 40 17.5 against
// 29.7, 256 of one 13.7 against 17.0.  Where A and B read once per 8 tokens
// outweigh that, the rule costs: n = 19456, k = 2560, rank 64, 64 tokens of one
// 22.6 against 20.0, 256 of 40 55.7 against 54.2, 256 of one 43.3 against 27.9.
constexpr int kLoraInBlock = 256;
constexpr int kLoraSmall = 8;      // tokens of a tile up to kLoraInBlock, and beyond
constexpr int kLoraTile = 32;
constexpr int kLoraMaxM = 4096;
constexpr int kPlanPerm = 4, kPlanTile = kPlanPerm + kLoraMaxM, kPlanInts = kPlanTile + 4 * kLoraMaxM;

__device__ __forceinline__ int32_t lora_adapter(const LoraParams& p, int t, bool& bad) {
  const int32_t a = p.adapter[t];
  bad = a >= p.n_adapters;
  return a < 0 || bad ? -1 : a;
}

// Grouping of more than kLoraInBlock tokens, by one block.  Tokens that come in
// long runs of one adapter (prompts; 16 tokens a run on average) stay in their
// order and each run makes tiles.  Others are sorted: a stable radix sort of
// (adapter, token) in shared memory, five bits a pass (40 adapters: two
// passes).  A warp takes 128 tokens in their order, 32 at a time; lanes with the
// same digit find one another by a match, so no atomics are needed and the
// order is always the same.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const __grid_constant__ LoraParams p) {
  __shared__ uint32_t key[2][kLoraMaxM];  // (adapter + 1) << 12 | token
  __shared__ int32_t count[32][33];       // [digit][warp]
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
  __syncthreads();
  int runs = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = i * 1024 + tid;
    runs += __syncthreads_count(t < p.m && (t == 0 || (key[0][t] >> 12) != (key[0][t - 1] >> 12)));
  }
  int cur = 0;
  const int bits = 32 - __clz(p.n_adapters + 1);  // so that the padding's bits are above all adapters'
  for (int shift = 12; shift < 12 + bits && runs * 16 > p.m; shift += 5) {
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
  {
    int32_t v = lane < warp ? warp_max[lane] : -1;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
    prev = max(prev, v);
  }
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
  int32_t total = warp_sum[lane], prior = lane < warp ? total : 0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, d);
    prior += __shfl_xor_sync(0xffffffffu, prior, d);
  }
  int32_t at_tile = incl - lead + prior;
  int32_t* first = reinterpret_cast<int32_t*>(key[cur ^ 1]);  // of each tile
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = i0 + i;
    if (at < p.m && (at - start[i]) % kLoraTile == 0) first[at_tile++] = at;
  }
  __syncthreads();
  for (int t = tid; t < total; t += 1024) {
    const int at = first[t], end = t + 1 < total ? first[t + 1] : p.m;
    reinterpret_cast<int4*>(p.plan + kPlanTile)[t] = make_int4(at, end - at, (int32_t)(key[cur][at] >> 12) - 1, 0);
  }
  if (tid == 0) p.plan[0] = total;
}

// 16 bytes of a row that is read on: two of its lines are fetched to L2 at the
// first (64 tokens 19.6 -> 18.5 us, 4096 tokens 71 -> 67 us).  STREAM: past L1,
// where nothing is read twice (64 tokens 17.2 us; with 32 tokens the other half
// of each line is wanted from L1: 59 against 49 us for 4096 tokens of A x).
// Not .nc: a block may start, and wait, while x or an adapter is still written.
template <bool STREAM>
__device__ __forceinline__ uint4 ldg16(const void* p) {
  uint4 v;
  if constexpr (STREAM)
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
  else
    asm volatile("ld.global.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
  return v;
}

// A x for NT columns of 8 tokens: this warp's sum over its pieces of k, to
// hp [16 ranks][8 NT].
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
  // The tensor core drops the bits below its accumulator's last place, so a
  // long chain of MMAs drifts (17408 features in one: 2.5e-6 of the result).
  // Every FLUSH rounds (16 to 24 MMAs) it is added to a sum of its own.
  constexpr int FLUSH = NT == 2 ? 2 : 4;
  float acc[NT][4], sum[NT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] = sum[nt][i] = 0.f;
  int round = 0;
  constexpr int U = NT == 4 ? 3 : (NT == 2 ? 4 : 2);  // pieces of 32 features in flight together
  for (int gi = g0; gi < g1; gi += U) {
    uint4 a[U][2], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t o = (int64_t)(gi + u < g1 ? gi + u : g1 - 1) * 32;
      a[u][0] = ldg16<NT == 1>(a0 + o);
      a[u][1] = ldg16<NT == 1>(a1 + o);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[u][nt] = ldg16<NT == 1>(xp[nt] + o);
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
    if (++round == FLUSH || gi + U >= g1) {
      round = 0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[nt][i] += acc[nt][i];
          acc[nt][i] = 0.f;
        }
    }
  }
  // [rank in tile][token]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    *reinterpret_cast<float2*>(hp + g * NT * 8 + nt * 8 + q * 2) = make_float2(sum[nt][0], sum[nt][1]);
    *reinterpret_cast<float2*>(hp + (g + 8) * NT * 8 + nt * 8 + q * 2) = make_float2(sum[nt][2], sum[nt][3]);
  }
}

// Step 3 for up to 8 tokens: this warp's groups of 32 features, e0, e0 + step,
// ... below e1, one at a time (B 32 ranks at a time, the next while these are
// multiplied).  One group and two pieces of A in step 1 leave registers for
// four blocks per SM: against two blocks with twice as much in flight each, 250
// tokens of 48 adapters 41 -> 30 us, 16 of 8 11.2 -> 10.7, 64 of 24 16.8 -> 17.4.
template <bool BF16, bool VEC>
__device__ __forceinline__ void lora_expand8(const LoraParams& p, int32_t ad, int e0, int e1, int step, const int32_t* tok,
                                             int cnt, const uint16_t* planes, int pstride, const float* mul) {
  constexpr int AHEAD = 2;
  constexpr int TERMS = BF16 ? 3 : 2;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  // MMA rows g, g + 8 of the two row tiles are features 4g .. 4g + 3
  const uint16_t* bp = static_cast<const uint16_t*>(p.b) + (int64_t)ad * p.n * p.rank + q * 4;
  for (int e = e0; e < e1; e += step) {
    const int f = e * 32 + 4 * g;
    uint2 b[AHEAD][4];
    auto load_b = [&](int r0) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int r = r0 + u * 16;
        const bool in = r + q * 4 < p.rank;  // false too in the last 8 of an odd number of eights
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[u][i] = in && f + i < p.n ? *reinterpret_cast<const uint2*>(bp + (int64_t)(f + i) * p.rank + r) : make_uint2(0, 0);
      }
    };
    load_b(0);
    float4 yv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = q * 2 + i;
      float4& v = yv[i];
      v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < cnt && f < p.n) {
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
    float acc[2][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][i] = 0.f;
    for (int r0 = 0; r0 < p.rank; r0 += 16 * AHEAD) {
      uint2 now[AHEAD][4];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) now[u][i] = b[u][i];
      if (r0 + 16 * AHEAD < p.rank) load_b(r0 + 16 * AHEAD);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int r = r0 + u * 16;
        if (r >= p.rank) break;
        const uint32_t m0[4] = {now[u][0].x, now[u][1].x, now[u][0].y, now[u][1].y};
        const uint32_t m1[4] = {now[u][2].x, now[u][3].x, now[u][2].y, now[u][3].y};
#pragma unroll
        for (int term = TERMS - 1; term >= 0; --term) {  // small terms first
          const uint2 h = *reinterpret_cast<const uint2*>(planes + (term * 8 + g) * pstride + r + q * 4);
          mma16<BF16>(acc[0], m0, h.x, h.y);
          mma16<BF16>(acc[1], m1, h.x, h.y);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = q * 2 + i;
      if (c >= cnt || f >= p.n) continue;
      const float s = mul[c];
      float4 v = yv[i];
      v.x = fmaf(acc[0][i], s, v.x);
      v.y = fmaf(acc[0][2 + i], s, v.y);
      v.z = fmaf(acc[1][i], s, v.z);
      v.w = fmaf(acc[1][2 + i], s, v.w);
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

// h of one token as terms of the operand type: lane l has ranks l, l + 32, ...
// in v; put(term, rank, bits) takes them.  Returns what the scaled terms are to
// be multiplied by.  Every term of an element has its sign and, unless the
// element is 0, is not 0 (all but the last are rounded down from below what is
// left of its size; fp16's are at least the smallest step, 2^-33 of the largest
// element), so that an infinite B gives its infinity, not 0 times infinity.
template <bool BF16, class Put>
__device__ __forceinline__ float lora_terms(float v[4], int ranks, Put put) {
  const int lane = threadIdx.x & 31;
  constexpr float BELOW = 0x1.fffffep-1f, STEP = 0x1p-24f;  // x * BELOW < x; fp16's smallest step
  float up = 1.f;
  if constexpr (!BF16) {
    float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    // the largest element goes to [2^9, 2^10); sums of fp16 products are below 2^64 or infinite
    const int e = min((int)((__float_as_uint(top) >> 23) & 255) - 127, 64);
    if (e > -110) {
      up = __uint_as_float((uint32_t)(e - 9 + 127) << 23);
      const float down = __uint_as_float((uint32_t)(9 - e + 127) << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] *= down;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = j * 32 + lane;
    if (r >= ranks) continue;
    constexpr int TERMS = BF16 ? 3 : 2;
    const uint16_t sign = (uint16_t)(__float_as_uint(v[j]) >> 16 & 0x8000u);
    const bool zero = v[j] == 0.f;
    float rest = fabsf(v[j]);
#pragma unroll
    for (int term = 0; term < TERMS; ++term) {
      const bool last = term == TERMS - 1;
      uint16_t t;
      float back;
      if constexpr (BF16) {
        t = last ? f_to_bf16_bits(rest) : (uint16_t)(__float_as_uint(rest * BELOW) >> 16);
        back = bf16_bits_to_f(t);
      } else {
        // two steps are left at least where there are three, so that the last term rounds to nearest
        const __half h = last ? __float2half_rn(rest) : __float2half_rz(fmaf(rest, BELOW, -2.f * STEP));
        t = !zero && !(h > __float2half_rn(0.f)) && rest == rest ? 1 : __half_as_ushort(h);
        back = __half2float(__ushort_as_half(t));
      }
      put(term, r, (uint16_t)(zero ? 0 : t | sign));
      if (rest < INFINITY) rest -= back;  // an infinity or NaN: all terms
    }
  }
  return up;
}

template <bool BF16, bool VEC>
__global__ void __cluster_dims__(LORA_CLUSTER, 1, 1) __launch_bounds__(LORA_THREADS, 4)
    lora_kernel(const __grid_constant__ LoraParams p) {
  constexpr int WARPS = LORA_THREADS / 32, COLS = kLoraSmall;
  constexpr int PSTRIDE = 128 + 16;  // a token's terms, 8 words past a multiple of 32 (no bank conflicts)
  __shared__ __align__(16) int32_t ids[kLoraInBlock];
  __shared__ int32_t tok[COLS], head[2], lead_count[WARPS];
  __shared__ float mul[COLS];
  __shared__ __align__(16) float h[128 * COLS], total[128 * COLS], hp[WARPS * 16 * COLS];  // [rank][token]
  __shared__ __align__(16) uint16_t planes[3 * COLS * PSTRIDE];                            // [term][token][rank]

  cg::cluster_group cluster = cg::this_cluster();
  const int part = cluster.block_rank();
  const int tile = blockIdx.x / LORA_CLUSTER;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  pdl_wait();
  pdl_launch_dependents();

  // ---- the tile's tokens: the tile-th token that is first of 8 of its adapter ---------
  int32_t id = -1;
  if (tid < p.m) {
    bool bad;
    id = lora_adapter(p, tid, bad);
    if (bad && blockIdx.x == 0) flag_bad_index(p.status);
  }
  ids[tid] = id;
  __syncthreads();
  int before = 0;  // tokens of the same adapter before this one
  if (tid < p.m) {
    const int4* v = reinterpret_cast<const int4*>(ids);
    for (int s = 0; s < tid; s += 4) {
      const int4 o = v[s >> 2];
      before += (o.x == id) + (s + 1 < tid && o.y == id) + (s + 2 < tid && o.z == id) + (s + 3 < tid && o.w == id);
    }
  }
  const bool lead = tid < p.m && before % COLS == 0;
  const uint32_t leads = __ballot_sync(0xffffffffu, lead);
  if (lane == 0) lead_count[warp] = __popc(leads);
  __syncthreads();
  int mine = __popc(leads & ((1u << lane) - 1)), tiles = 0;
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) mine += lead_count[w];
    tiles += lead_count[w];
  }
  if (tile >= tiles) return;  // the whole cluster
  if (lead && mine == tile) {
    head[0] = id;
    head[1] = before;
  }
  __syncthreads();
  const int32_t ad = head[0];
  const bool in = tid < p.m && id == ad && before >= head[1] && before < head[1] + COLS;
  if (in) tok[before - head[1]] = tid;
  const int cnt = __syncthreads_count(in);

  if (ad < 0) {  // no adapter: y as it is
    if (p.out != p.y)
      for (int c = 0; c < cnt; ++c) {
        const float* src = p.y + tok[c] * p.y_stride;
        float* dst = p.out + tok[c] * p.out_stride;
        const int quads = VEC ? p.n >> 2 : 0;
        for (int i = part * LORA_THREADS + tid; i < quads; i += LORA_CLUSTER * LORA_THREADS)
          reinterpret_cast<float4*>(dst)[i] = reinterpret_cast<const float4*>(src)[i];
        for (int i = quads * 4 + part * LORA_THREADS + tid; i < p.n; i += LORA_CLUSTER * LORA_THREADS) dst[i] = src[i];
      }
    return;
  }

  // ---- 1. h = A x over this block's share of k -----------------------------------
  const int rts = (p.rank + 15) >> 4;  // 16-row tiles of A
  const int kparts = WARPS / rts;      // warps that share a tile's k
  const int rt = warp / kparts, kp = warp - rt * kparts;
  if (rt < rts) {
    const int pieces = p.k >> 5, shares = LORA_CLUSTER * kparts, s = part * kparts + kp;
    const int g0 = (int)((int64_t)pieces * s / shares), g1 = (int)((int64_t)pieces * (s + 1) / shares);
    lora_shrink<BF16, 1>(p, ad, rt, tok, cnt, g0, g1, hp + warp * 16 * COLS);
  }
  __syncthreads();
  for (int i = tid; i < p.rank * COLS; i += LORA_THREADS) {
    const float* src = hp + (i / (16 * COLS)) * kparts * 16 * COLS + i % (16 * COLS);
    float s = 0.f;
    for (int w = 0; w < kparts; ++w) s += src[w * 16 * COLS];
    h[i] = s;
  }
  cluster.sync();

  // ---- 2. the cluster's sum, as terms of the operand type --------------------------
  for (int i = tid; i < p.rank * COLS / 4; i += LORA_THREADS) {
    float4 v[LORA_CLUSTER];
#pragma unroll
    for (int b = 0; b < LORA_CLUSTER; ++b) v[b] = reinterpret_cast<const float4*>(cluster.map_shared_rank(h, b))[i];
#pragma unroll
    for (int b = 1; b < LORA_CLUSTER; ++b) v[0].x += v[b].x, v[0].y += v[b].y, v[0].z += v[b].z, v[0].w += v[b].w;
    reinterpret_cast<float4*>(total)[i] = v[0];
  }
  __syncthreads();
  {
    const int c = warp;  // a warp per token
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = j * 32 + lane;
      v[j] = r < p.rank && c < cnt ? total[r * COLS + c] : 0.f;
    }
    const float up = lora_terms<BF16>(v, rts * 16, [&](int term, int r, uint16_t t) { planes[(term * COLS + c) * PSTRIDE + r] = t; });
    if (lane == 0) mul[c] = up * (p.scale ? p.scale[ad] : 1.f);
  }
  __syncthreads();

  // ---- 3. out = y + s B h over this block's share of n -------------------------------
  const int groups = (p.n + 31) >> 5;
  const int e0 = (int)((int64_t)groups * part / LORA_CLUSTER) + warp;
  const int e1 = (int)((int64_t)groups * (part + 1) / LORA_CLUSTER);
  lora_expand8<BF16, VEC>(p, ad, e0, e1, WARPS, tok, cnt, planes, PSTRIDE, mul);
  cluster.sync();  // the other blocks have read this one's h
}

// ---- more than kLoraInBlock tokens -------------------------------------------------

// h of the plan's tiles, split over k.  Blocks take (tile, split) in turn; the
// warps of a block split the piece of k (and the 16-row tiles of A), so that x
// comes from memory once and A once per 32 tokens.  The last split of a tile to
// arrive adds all of them, in their order, and leaves the operand terms.
template <bool BF16>
__global__ void __launch_bounds__(LORA_THREADS, 2) lora_shrink_kernel(const __grid_constant__ LoraParams p) {
  constexpr int WARPS = LORA_THREADS / 32, TERMS = BF16 ? 3 : 2;
  __shared__ int32_t tok[kLoraTile], last;
  __shared__ __align__(16) float hp[WARPS * 16 * kLoraTile];
  __shared__ float h[kLoraTile * 129];  // [token][rank], odd stride
  // While the tokens are still being grouped: the first 8 MB of x to L2 (what
  // comes from memory in that time; 1000 tokens 57.6 -> 56.1 us, 4096 tokens
  // 67.6 -> 67.0, with 24 MB 68.1).
  const int64_t kbs = (int64_t)p.m * (p.k >> 9);  // of 512 features
  for (int64_t c = blockIdx.x * LORA_THREADS + threadIdx.x; c < (kbs < 8192 ? kbs : 8192); c += gridDim.x * LORA_THREADS)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(static_cast<const uint8_t*>(p.x) + c * 1024),
                 "r"(1024u));
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = p.plan[0] * p.splits;
  const int rts = (p.rank + 15) >> 4, kparts = WARPS / rts;
  const int rt = warp / kparts, kp = warp - rt * kparts;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int tile = u / p.splits, split = u - tile * p.splits;
    const int4 info = reinterpret_cast<const int4*>(p.plan + kPlanTile)[tile];
    const int i0 = info.x, cnt = info.y, ad = info.z;
    if (ad < 0) continue;
    __syncthreads();  // the previous unit's sums and tokens are read
    if (tid < cnt) tok[tid] = p.plan[kPlanPerm + i0 + tid];
    __syncthreads();
    const int cols = cnt <= 8 ? 8 : (cnt <= 16 ? 16 : 32);
    if (rt < rts) {
      const int pieces = p.k >> 5, shares = p.splits * kparts, s = split * kparts + kp;
      const int g0 = (int)((int64_t)pieces * s / shares), g1 = (int)((int64_t)pieces * (s + 1) / shares);
      float* to = hp + warp * 16 * kLoraTile;
      if (cols == 8)
        lora_shrink<BF16, 1>(p, ad, rt, tok, cnt, g0, g1, to);
      else if (cols == 16)
        lora_shrink<BF16, 2>(p, ad, rt, tok, cnt, g0, g1, to);
      else
        lora_shrink<BF16, 4>(p, ad, rt, tok, cnt, g0, g1, to);
    }
    __syncthreads();
    // lanes are tokens, warps ranks
    float* part = p.h + (int64_t)i0 * p.rank;
    const int64_t step = (int64_t)p.m * p.rank;  // between splits
    if (lane < cnt) {
#pragma unroll 4
      for (int r = warp; r < p.rank; r += WARPS) {
        const float* src = hp + (r >> 4) * kparts * 16 * kLoraTile + (r & 15) * cols + lane;
        float sum = 0.f;
        for (int w = 0; w < kparts; ++w) sum += src[w * 16 * kLoraTile];
        if (p.splits == 1)
          h[lane * 129 + r] = sum;
        else
          part[split * step + r * cnt + lane] = sum;
      }
    }
    if (p.splits > 1) {
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        last = atomicAdd(p.counters + tile, 1) == p.splits - 1;
        if (last) p.counters[tile] = 0;
        __threadfence();
      }
      __syncthreads();
      if (!last) continue;
      if (lane < cnt) {
#pragma unroll 2
        for (int r = warp; r < p.rank; r += WARPS) {
          float v[8];
#pragma unroll
          for (int sp = 0; sp < 8; ++sp) v[sp] = sp < p.splits ? __ldcg(part + sp * step + r * cnt + lane) : 0.f;
          h[lane * 129 + r] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
      }
    }
    __syncthreads();
    for (int c = warp; c < cnt; c += WARPS) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = j * 32 + lane < p.rank ? h[c * 129 + j * 32 + lane] : 0.f;
      uint16_t* to = p.terms + (int64_t)(i0 + c) * 3 * p.rank;
      const float up = lora_terms<BF16>(v, p.rank, [&](int term, int r, uint16_t t) { to[term * p.rank + r] = t; });
      if (lane == 0) p.mul[i0 + c] = up * (p.scale ? p.scale[ad] : 1.f);
    }
    static_assert(TERMS <= 3, "terms");
  }
}

// Shared memory of the second product's blocks; PANELS of 64 ranks.
template <int PANELS>
struct LoraSmem {
  static constexpr int BUFS = PANELS == 1 ? 3 : 2;  // tiles of B in flight or in use
  static constexpr int PANEL_B = 128 * 128;         // 128 features x 64 ranks
  static constexpr int PANEL_H = kLoraTile * 128;   // 32 tokens x 64 ranks
  uint8_t b[BUFS][PANELS * PANEL_B];
  uint8_t terms[3][PANELS * PANEL_H];
  // of the tokens: rows of y and out (elements), and what their sums are multiplied by
  alignas(16) uint32_t yoff[kLoraTile];
  alignas(16) uint32_t ooff[kLoraTile];
  alignas(16) float mul[kLoraTile];
  uint64_t bar[2];
  uint32_t tmem;
};

// out = y + s B h: D [128 features][32 tokens] = B [128][rank] (terms of h)^T
// on the tcgen05 tensor cores.  The (tile, 128 features) units, in tile order,
// are split evenly over the blocks.  While a tile is finished (accumulator and
// y to out) the next is multiplied and the one after it copied; its y is loaded
// a tile ahead too.  A thread has one feature and 16 tokens, so a warp's
// accesses of y and out are 128 bytes in a row at any alignment.
template <bool BF16, int PANELS>
__global__ void __launch_bounds__(LORA_THREADS, PANELS == 1 ? 3 : 2) lora_expand_kernel(const __grid_constant__ LoraParams p) {
  using S = LoraSmem<PANELS>;
  constexpr int TERMS = BF16 ? 3 : 2, BUFS = S::BUFS;
  constexpr uint32_t IDESC = (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | ((kLoraTile >> 3) << 17) | ((128 >> 4) << 24);
  constexpr int COLS = kLoraTile / 2;  // tokens of a thread
  extern __shared__ __align__(16) uint8_t smem[];
  S& sm = *reinterpret_cast<S*>(smem + (-smem_u32(smem) & 1023u));  // the operand tiles are aligned to 1 KB
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t bar = smem_u32(sm.bar);

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  pdl_wait();
  // tensor memory only from here on (the kernel before may still be waiting for
  // its own until it has ended), and the next kernel only after it (so that it
  // cannot take this block's and then wait for it)
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sm.tmem)), "r"(64u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = sm.tmem;

  const int steps = (p.rank + 15) >> 4, fbs = (p.n + 127) >> 7;
  const int c0 = (warp >> 2) * COLS, row = (warp & 3) * 32 + lane;
  const int64_t units = (int64_t)p.plan[0] * fbs;
  int64_t u = units * blockIdx.x / gridDim.x;
  const int64_t u_end = units * (blockIdx.x + 1) / gridDim.x;
  int it = 0;  // products issued by this block, modulo 4
  while (u < u_end) {
    const int tile = (int)(u / fbs), t0 = (int)(u - (int64_t)tile * fbs);
    const int t1 = u_end - u < fbs - t0 ? t0 + (int)(u_end - u) : fbs;
    u += t1 - t0;
    const int4 info = reinterpret_cast<const int4*>(p.plan + kPlanTile)[tile];
    const int i0 = info.x, cnt = info.y, ad = info.z;
    if (ad < 0 && p.out == p.y) continue;
    __syncthreads();  // the previous tile's offsets, terms and products are done with
    if (tid < kLoraTile) {  // tokens that are not there: row 0, never written
      const int32_t t = tid < cnt ? p.plan[kPlanPerm + i0 + tid] : 0;
      sm.yoff[tid] = (uint32_t)t * (uint32_t)p.y_stride;
      sm.ooff[tid] = (uint32_t)t * (uint32_t)p.out_stride;
    }
    if (ad < 0) {  // no adapter: y as it is
      __syncthreads();
      for (int t = t0; t < t1; ++t) {
        const int f = t * 128 + row;
        if (f >= p.n) continue;
        float v[COLS];
#pragma unroll
        for (int j = 0; j < COLS; ++j) v[j] = p.y[sm.yoff[c0 + j] + f];
#pragma unroll
        for (int j = 0; j < COLS; ++j)
          if (c0 + j < cnt) p.out[sm.ooff[c0 + j] + f] = v[j];
      }
      continue;
    }
    // rows of 64 ranks are 128 bytes, 16-byte chunk i of row r at i ^ (r & 7)
    // (the 128-byte swizzle); ranks up to the last step of 16 that are not
    // there are zeros.  This thread copies chunk tid % 8 of every 32nd row.
    const int ch = tid & 7, rw = tid >> 3;
    const uint16_t* bsrc = static_cast<const uint16_t*>(p.b) + ((int64_t)ad * p.n + rw) * p.rank + ch * 8;
    const uint32_t bdst = smem_u32(sm.b[0]) + rw * 128 + ((ch ^ (rw & 7)) << 4);
    auto fetch = [&](int t, int buf) {
      if (t < t1) {
#pragma unroll
        for (int pn = 0; pn < PANELS; ++pn) {
          const int r = pn * 64 + ch * 8;
          if (r >= steps * 16) continue;
          const uint16_t* src = bsrc + (int64_t)t * 128 * p.rank + pn * 64;
          const uint32_t dst = bdst + (buf * PANELS + pn) * S::PANEL_B;
          if (t * 128 + 128 <= p.n && r < p.rank) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async16(dst + i * 32 * 128, src + i * 32 * p.rank, true);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool in = t * 128 + i * 32 + rw < p.n && r < p.rank;
              cp_async16(dst + i * 32 * 128, in ? src + i * 32 * p.rank : static_cast<const uint16_t*>(p.b), in);
            }
          }
        }
      }
      cp_async_commit();
    };
    float yv[COLS];
    auto load_y = [&](int t) {
      const int f = t * 128 + row;
      if (t < t1 && f < p.n) {
        // (tokens that are not there read row 0's y)
#pragma unroll
        for (int j = 0; j < COLS; j += 4) {
          const uint4 o = *reinterpret_cast<const uint4*>(sm.yoff + c0 + j);
          yv[j] = p.y[o.x + f], yv[j + 1] = p.y[o.y + f], yv[j + 2] = p.y[o.z + f], yv[j + 3] = p.y[o.w + f];
        }
      }
    };
    // the lines of y three tiles ahead: to L2, so that load_y finds them there
    auto prefetch_y = [&](int t) {
      const int c = tid >> 2, f = t * 128 + (tid & 3) * 32;
      if (tid < 4 * kLoraTile && t < t1 && c < cnt && f < p.n)
        asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p.y + sm.yoff[c] + f));
    };
    auto multiply = [&](int buf) {  // one thread; small terms first, since each sum loses the bits below its last place
      tc_fence_after();
      const uint32_t d = tmem + (it & 1) * kLoraTile;
#pragma unroll
      for (int term = TERMS - 1; term >= 0; --term)
        for (int k = 0; k < steps; ++k)
          umma_f16(d, umma_smem_desc(smem_u32(sm.b[buf]) + (k >> 2) * S::PANEL_B + (k & 3) * 32),
                   umma_smem_desc(smem_u32(sm.terms[term]) + (k >> 2) * S::PANEL_H + (k & 3) * 32), IDESC,
                   term < TERMS - 1 || k > 0);
      umma_commit(bar + 8 * (it & 1));
    };
    // the operand terms of the tokens (zeros for those that are not there), 8 ranks at a time
    for (int i = tid; i < TERMS * kLoraTile * 8 * PANELS; i += LORA_THREADS) {
      const int hc = i & 7, c = (i >> 3) & (kLoraTile - 1), tp = i / (8 * kLoraTile), term = tp % TERMS, pn = tp / TERMS;
      const int r = pn * 64 + hc * 8;
      if (r < steps * 16) {
        const bool in = c < cnt && r < p.rank;
        cp_async16(smem_u32(sm.terms[term]) + pn * S::PANEL_H + c * 128 + ((hc ^ (c & 7)) << 4),
                   in ? p.terms + ((int64_t)(i0 + c) * 3 + term) * p.rank + r : p.terms, in);
      }
    }
    if (tid < kLoraTile) sm.mul[tid] = tid < cnt ? p.mul[i0 + tid] : 0.f;
    fetch(t0, 0);
    fetch(t0 + 1, 1);
    __syncthreads();  // the tokens' rows
    load_y(t0);
    prefetch_y(t0 + 1);
    prefetch_y(t0 + 2);
    cp_async_wait<1>();
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) multiply(0);
    int buf = 0;
    for (int t = t0; t < t1; ++t) {
      // here the product of tile t is under way and the copies of t + 1 are issued
      const int nbuf = buf + 1 == BUFS ? 0 : buf + 1, fbuf = buf == 0 ? BUFS - 1 : buf - 1;
      const uint32_t d = tmem + (it & 1) * kLoraTile, mybar = bar + 8 * (it & 1), parity = (it >> 1) & 1;
      it = (it + 1) & 3;
      bool good = true;
      if constexpr (BUFS == 2) good = mbar_wait(mybar, parity, 1u << 21);  // the buffer to be filled is this product's
      else fetch(t + BUFS - 1, fbuf);  // the buffer of tile t - 1, whose product every thread has waited for
      if constexpr (BUFS == 3) {
        if (t + 1 < t1) {
          cp_async_wait<1>();
          fence_async_smem();
          tc_fence_before();
          __syncthreads();
          if (tid == 0) multiply(nbuf);
        }
      }
      float v[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) v[j] = yv[j];
      load_y(t + 1);
      prefetch_y(t + 3);
      if constexpr (BUFS == 3) good = mbar_wait(mybar, parity, 1u << 21);
      // a wait that runs out (it cannot in a healthy launch) leaves the outputs undefined and says so
      good = __all_sync(0xffffffffu, good);
      if (!good && lane == 0) atomicExch(p.status, UM_TIMEOUT_STATUS);
      if constexpr (BUFS == 2) {
        fetch(t + 2, buf);
        if (t + 1 < t1) {
          cp_async_wait<1>();
          fence_async_smem();
          tc_fence_before();
          __syncthreads();
          if (tid == 0) multiply(nbuf);
        }
      }
      buf = nbuf;
      if (!good) continue;
      tc_fence_after();
      uint32_t acc[COLS];
      tmem_ld16(d + ((uint32_t)((warp & 3) * 32) << 16) + c0, acc);
      const int f = t * 128 + row;
      if (f < p.n) {
#pragma unroll
        for (int j = 0; j < COLS; j += 4) {
          const uint4 o = *reinterpret_cast<const uint4*>(sm.ooff + c0 + j);
          const float4 m = *reinterpret_cast<const float4*>(sm.mul + c0 + j);
          const float r0 = fmaf(__uint_as_float(acc[j]), m.x, v[j]), r1 = fmaf(__uint_as_float(acc[j + 1]), m.y, v[j + 1]);
          const float r2 = fmaf(__uint_as_float(acc[j + 2]), m.z, v[j + 2]), r3 = fmaf(__uint_as_float(acc[j + 3]), m.w, v[j + 3]);
          if (c0 + j + 4 <= cnt) {
            p.out[o.x + f] = r0, p.out[o.y + f] = r1, p.out[o.z + f] = r2, p.out[o.w + f] = r3;
          } else {
            if (c0 + j < cnt) p.out[o.x + f] = r0;
            if (c0 + j + 1 < cnt) p.out[o.y + f] = r1;
            if (c0 + j + 2 < cnt) p.out[o.z + f] = r2;
          }
        }
      }
    }
    cp_async_wait<0>();
    tc_fence_before();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(64u));
  }
}

}  // namespace tq
