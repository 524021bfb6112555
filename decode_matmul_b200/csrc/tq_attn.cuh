// tq_attn.cuh -- attention of new tokens over the paged key/value cache.
//
// Per row and query head: o = sum_j softmax_j(c q.k_j) v_j over the visible
// keys, in one pass with the running maximum M and sum L of the softmax
// (weights 2^(s - M), s = c log2(e) q.k; M rises: O and L are scaled by
// 2^(M_old - M_new)).
//
// Bound: the bytes of the cache, each read once; the query heads that share a
// key head share its tiles.  A tile is 16 or 32 keys of one (row, key head,
// group of up to 8 or 16 query heads).  All tiles of the call, in row-major order, are
// split evenly over the blocks and in each block over its warps, whatever the
// rows' lengths are (the lengths are read on the device, so a captured call
// serves any).  Each warp streams its tiles through a ring of its own in
// shared memory (16-byte asynchronous copies; no barrier between warps), and
// computes
//   S^T = K Q^T   (m16n8k16: 16 keys x 8 heads)
//   O^T += V^T P^T  (16 features x 8 heads per MMA)
// so that the 8-wide side of the MMA is the heads and none of the 16-wide
// side is padding; P^T's operand layout is the transpose of S^T's result
// layout (movmatrix).  Warp MMAs suffice: at the cache's bandwidth they need
// a fifth (bf16) to a quarter (e4m3) of their rate, and the one-row-per-key
// layout they take needs no tensor map, so any page size and strides work.
// Items (row, key head, head group) that a warp holds whole are written by
// it.  The others leave partial (O, M, L), joined first inside the block, then
// over the blocks by the last to arrive, in a fixed order (the same bits on
// every run).
// Head and tail (stamped on the GPU): the split takes 1.2 us, page look-ups and
// the first tile 1.5 us (4 us from HBM), the joins 2 to 5 us; between them the
// warps stream at 7 TB/s.  Measured, three caches in turn: 64 rows of 3 to 8192
// keys, 8 heads x 128 bf16: 72 us, 5.2 TB/s; 16 rows of 20000 to 65536 e4m3
// keys: 262 us, 5.2 TB/s (0.44 instructions per scheduler and cycle from two
// warps: their own latencies bound it); one row of 777 keys: 10 us.
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
  int32_t group;        // query heads per key head
  int32_t head_groups;  // items per key head
  int32_t team;         // warps that work on neighbouring items over the same keys
  int32_t min_units;    // units a block takes at least before another is used
  uint32_t page_mul, page_shift;  // j / page_size = (umulhi(j, mul) + j) >> shift
  // the cache's strides in units of unit bytes (a power of two that divides
  // them all), in which every offset fits 32 bits
  uint32_t unit, page_step, token_step, head_step;
  float scale;
  int32_t out_bf16;
  int32_t* counters;
  float* partials;  // [grid][2][kTeamMax][AttnCfg::PART]
  int32_t* status;
};

template <int T, int D, int NT>
struct AttnCfg {
  static constexpr int EB = KvElem<T>::bytes;
  static constexpr int RB = D * EB;          // bytes of a key
  static constexpr int CPR = RB / 16;        // 16-byte chunks of a key
  // keys of a tile: 32 where 64 KB of ring per 8 warps then still hold it
  // (longer independent chains per step), else 16
  static constexpr int TK = RB <= 128 ? 32 : 16;
  static constexpr int KT = TK / 16;
  static constexpr int STAGE = 2 * TK * RB;  // the keys, then the values
  static constexpr int COLS = 8 * NT;        // head columns
  static constexpr int PART = D * COLS + 2 * COLS;  // floats of a partial: O [D][COLS], M, L
  static constexpr int SLOT = PART * 4;
  static constexpr int CTL = 2048;
  static constexpr int fit(int warps) { return ((227 * 1024 - CTL) / warps - SLOT) / STAGE; }
  // as many warps as leave each a ring of three tiles, else four
  static constexpr int WARPS = fit(8) >= 3 ? 8 : (fit(6) >= 3 ? 6 : 4);
  static constexpr int STAGES = fit(WARPS) > 3 ? 3 : fit(WARPS);
  static constexpr int RING = STAGES * STAGE > SLOT ? STAGES * STAGE : SLOT;  // the tail's partial reuses the ring
  static constexpr int WARP_BYTES = RING + SLOT;
  static constexpr int SMEM = WARPS * WARP_BYTES + CTL;
  static constexpr int THREADS = WARPS * 32;
  // Chunk ch of key row r lies at chunk ch ^ swz(r) of its row, so that the
  // same chunk of 8 rows in a row (one ldmatrix phase) is in 8 different
  // 16-byte banks; the xor stays inside aligned groups, so rows of any of
  // these sizes map onto themselves.
  static __host__ __device__ constexpr int swz(int r) {
    return CPR % 8 == 0 ? (r & 7) : (CPR % 4 == 0 ? ((r >> 1) & 3) : ((r >> 2) & 1));
  }
  static_assert(CPR % 8 == 0 || CPR == 4 || CPR == 12 || CPR == 6, "row sizes the swizzle covers");
  static_assert(STAGES >= 2 && SMEM <= 227 * 1024 && WARP_BYTES % 16 == 0, "ring");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// the four e4m3 values of a word as two fp16 pairs (exact)
__device__ __forceinline__ void e4m3x4_to_h2(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }\n"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
template <bool BF16>
__device__ __forceinline__ void mma16(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma_16816(c, a, b0, b1);
}

// The weights of the second product as MMA operands.  They are at most 2^UP and
// the sum of a weight's terms (each word has those of two weights) keeps
// binary32 accuracy: three bf16 terms (24 bits) or two fp16 terms (22 bits).
// UP = 15 for fp16: its smallest step, 2^-24, then is 2^-39 of the largest
// weight; with weights of at most 1 a key of less than 2^-25 would add nothing
// to O while the sum of the weights still counted it (16384 keys 18 below one
// key in e^s: all of their part of the output lost).  O and the sum carry the
// same 2^UP, which cancels.
// With one fp16 term (2^-12) or two of bf16 (2^-17) 6 to 10%, or 0.2%, of the bf16
// outputs were rounded to the other neighbour.
// For 16-bit caches every term of a weight is positive: an infinite value then
// gives its infinity, where a term of 0 or of the other sign would make it NaN.
// So all terms but the last are rounded down from below what is left of the
// weight.  fp16's are at least its smallest step, so weights below 2^-38 of the
// largest count as that much (hidden keys too: their values are zeros).
template <int T>
struct AttnWeights {
  static constexpr int TERMS = T == KV_BF16 ? 3 : 2;
  static constexpr float UP = T == KV_BF16 ? 0.f : 15.f;
  static constexpr float BELOW = 0x1.fffffep-1f;  // x * BELOW < x in binary32 (by one step, or half of one)
  static __device__ __forceinline__ void split(float a, float b, uint32_t t[TERMS]) {
    if constexpr (T == KV_BF16) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t ha = __float_as_uint(a * BELOW), hb = __float_as_uint(b * BELOW);
        t[k] = __byte_perm(ha, hb, 0x7632);
        a -= __uint_as_float(ha & 0xffff0000u);
        b -= __uint_as_float(hb & 0xffff0000u);
      }
      t[2] = KvElem<KV_BF16>::pack2(a, b);
    } else {
      constexpr float STEP = 0x1p-24f;  // two of them are left at least where there are three, so that t[1] rounds to nearest
      if constexpr (T == KV_F16) {
        asm("cvt.rz.f16x2.f32 %0, %1, %2;\n" : "=r"(t[0]) : "f"(fmaf(b, BELOW, -2 * STEP)), "f"(fmaf(a, BELOW, -2 * STEP)));
        t[0] = max_h2(t[0], 0x00010001u);
      } else {
        t[0] = f2_to_h2(a, b);
      }
      const float2 f = h2_to_f2(t[0]);
      t[1] = f2_to_h2(a - f.x, b - f.y);
      if constexpr (T == KV_F16) t[1] = max_h2(t[1], 0x00010001u);
    }
  }
  static __device__ __forceinline__ uint32_t max_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
};

// The visible keys of a row.
struct AttnRow {
  int32_t keys, first, seq;  // how many, the first of them, block-table row
  // tiles of an item of the row: at least one, so that rows without keys are written too
  template <int TK>
  __device__ __forceinline__ int32_t tiles() const {
    return keys > 0 ? (int32_t)(((uint32_t)keys + TK - 1) / TK) : 1;
  }
};

// An item of n tiles takes n + kItemCost units of the split: its start and end
// (queries, partial or final output) cost about as much as four tiles, which
// would leave the blocks that hold many short rows behind (64 rows of 3 to
// 8192 keys: the slowest block took 1.35 times the mean without it).
constexpr int kItemCost = 4;

// Items next to each other in a row can be worked on by a team of warps, one
// item each over the same keys: where a key of one head is less than 256 bytes
// and its neighbours are other heads' (16 rows of 20000 to 65536 e4m3 keys of
// 8 x 128 bytes: 268 us one by one, the same with the heads apart in memory
// 219 us), and for two groups of query heads on one key head.
constexpr int kTeamMax = 4;
constexpr int kTeamUnits = 100;  // units per block from which teams are formed

// Where a warp stands in the tile order (an item here is a team's items).
struct AttnWalk {
  int32_t row_at;        // first unit of the row in the whole call's order
  int32_t row, item, j;  // row, item in the row, tile in the item
  int32_t n;             // tiles of an item of this row
  AttnRow r;
};

// bad: the row's sequence or position is outside the block table
__device__ __forceinline__ AttnRow attn_row(const AttnParams& p, int row, bool& bad) {
  AttnRow r;
  const int32_t pos = p.pos[row];
  r.seq = p.seq ? p.seq[row] : row;
  bad = pos >= 0 && (r.seq < 0 || r.seq >= p.c.n_seqs || pos >= p.c.page_size * p.c.max_pages);
  r.first = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
  r.keys = pos < 0 || bad ? 0 : pos - r.first + 1;
  return r;
}

// ---- join -----------------------------------------------------------------------
// A part is (O, M, L) relative to its own maximum: O [D][COLS], M [COLS],
// L [COLS].  Parts join to sum_i 2^(M_i - M) O_i.  When its warps are done a
// block joins their parts of each item in shared memory.  Of an item that goes
// beyond the block (at most its first and its last per team member) it
// publishes the result, and the last block to publish joins the blocks' parts,
// in groups of kJoin when there are more, so that a row spread over the whole
// GPU takes two short rounds.  No block waits for another.
constexpr int kJoin = 16;
constexpr int kTopCounters = 4096;  // counters of the second round (the first's are 2 kTeamMax per block)

// The joined parts of one thread: QPT quads of O at quad u * THREADS + tid,
// all of the same four columns col.
template <int D, int COLS, int THREADS>
struct AttnSum {
  static constexpr int QUADS = D * COLS / 4;
  static constexpr int QPT = (QUADS + THREADS - 1) / THREADS;
  static constexpr bool FULL = QUADS % THREADS == 0;
  static_assert((THREADS * 4) % COLS == 0, "columns");
  float4 acc[QPT];
  float M[4], L[4];

  static __device__ __forceinline__ float weight(float m, float top) { return top == -INFINITY ? 0.f : ex2(m - top); }
  static __device__ __forceinline__ int col() { return (threadIdx.x * 4) % COLS; }
  static __device__ __forceinline__ bool in(int u) { return FULL || u * THREADS + (int)threadIdx.x < QUADS; }
  static __device__ __forceinline__ int quad(int u) { return (u * THREADS + threadIdx.x) * 4; }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 4; ++k) M[k] = -INFINITY, L[k] = 0.f;
#pragma unroll
    for (int u = 0; u < QPT; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // raises the maxima to cover m, scaling what has been summed
  __device__ __forceinline__ void raise(float4 m) {
    const float f[4] = {fmaxf(M[0], m.x), fmaxf(M[1], m.y), fmaxf(M[2], m.z), fmaxf(M[3], m.w)};
    float r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      r[k] = weight(M[k], f[k]);
      M[k] = f[k];
      L[k] *= r[k];
    }
#pragma unroll
    for (int u = 0; u < QPT; ++u) acc[u].x *= r[0], acc[u].y *= r[1], acc[u].z *= r[2], acc[u].w *= r[3];
  }
  // B parts at p(0) .. p(B-1), of which the first n count: their loads are in flight together
  template <int B, class P>
  __device__ __forceinline__ void add(int n, P p) {
    float4 m[B], l[B], v[B][QPT];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      m[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < n) {
        const float* src = p(i);
        m[i] = *reinterpret_cast<const float4*>(src + D * COLS + col());
        l[i] = *reinterpret_cast<const float4*>(src + D * COLS + COLS + col());
#pragma unroll
        for (int u = 0; u < QPT; ++u)
          if (in(u)) v[i][u] = *reinterpret_cast<const float4*>(src + quad(u));
      }
    }
    float4 top = m[0];
#pragma unroll
    for (int i = 1; i < B; ++i)
      top = make_float4(fmaxf(top.x, m[i].x), fmaxf(top.y, m[i].y), fmaxf(top.z, m[i].z), fmaxf(top.w, m[i].w));
    raise(top);
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (i < n) {
        const float f[4] = {weight(m[i].x, M[0]), weight(m[i].y, M[1]), weight(m[i].z, M[2]), weight(m[i].w, M[3])};
        L[0] += f[0] * l[i].x, L[1] += f[1] * l[i].y, L[2] += f[2] * l[i].z, L[3] += f[3] * l[i].w;
#pragma unroll
        for (int u = 0; u < QPT; ++u)
          if (in(u))
            acc[u].x += f[0] * v[i][u].x, acc[u].y += f[1] * v[i][u].y, acc[u].z += f[2] * v[i][u].z,
                acc[u].w += f[3] * v[i][u].w;
      }
  }
  // n blocks' parts at p(0) .. p(n-1)
  template <class P>
  __device__ __forceinline__ void sum(int n, P p) {
    constexpr int B = QPT == 1 ? 8 : (QPT <= 4 ? 4 : 2);
    clear();
#pragma unroll 1
    for (int i = 0; i < n; i += B) add<B>(n - i, [&](int k) { return p(i + k); });
  }
  __device__ __forceinline__ void store(float* to) const {
#pragma unroll
    for (int u = 0; u < QPT; ++u)
      if (in(u)) *reinterpret_cast<float4*>(to + quad(u)) = acc[u];
    if (threadIdx.x < COLS / 4) {
      *reinterpret_cast<float4*>(to + D * COLS + col()) = make_float4(M[0], M[1], M[2], M[3]);
      *reinterpret_cast<float4*>(to + D * COLS + COLS + col()) = make_float4(L[0], L[1], L[2], L[3]);
    }
  }
  // the item's rounded output
  __device__ __forceinline__ void write(const AttnParams& p, int row, int item) const {
    const int kvh = item / p.head_groups, h0 = (item - kvh * p.head_groups) * COLS + col();
    const float vsc = p.c.vs ? p.c.vs[kvh] : 1.f;
    uint16_t* out = static_cast<uint16_t*>(p.out) + ((int64_t)row * p.q_heads + kvh * p.group + h0) * D;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (h0 + k >= p.group) continue;
      const float inv = L[k] == 0.f ? 0.f : vsc / L[k];
#pragma unroll
      for (int u = 0; u < QPT; ++u)
        if (in(u)) {
          const float y = (k == 0 ? acc[u].x : k == 1 ? acc[u].y : k == 2 ? acc[u].z : acc[u].w) * inv;
          out[k * D + quad(u) / COLS] = p.out_bf16 ? f_to_bf16_bits(y) : __half_as_ushort(__float2half_rn(y));
        }
    }
  }
};

template <int TK>
__device__ __forceinline__ void attn_next(const AttnParams& p, AttnWalk& w, int items) {
  if (++w.j < w.n) return;
  w.j = 0;
  if (++w.item < items) return;
  w.item = 0;
  w.row_at += (w.n + kItemCost) * items;
  if (++w.row < p.m) {
    bool bad;
    w.r = attn_row(p, w.row, bad);
    w.n = w.r.tiles<TK>();
  }
}

template <int T, int D, int NT>
__global__ void __launch_bounds__(AttnCfg<T, D, NT>::THREADS, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  using C = AttnCfg<T, D, NT>;
  constexpr bool BF = T == KV_BF16;
  constexpr bool F8 = T == KV_E4M3;
  constexpr int W = C::WARPS, S = C::STAGES, COLS = C::COLS, MT = D / 16, TK = C::TK, KT = C::KT;
  constexpr int TERMS = AttnWeights<T>::TERMS;
  extern __shared__ __align__(16) uint8_t smem[];
  struct Part {  // what a warp left in a slot
    int32_t first, n, row, item;  // unit of the item's first tile, its tiles (0: nothing)
    int32_t member;
  };
  struct Ctl {
    int64_t warp_sum[W];
    AttnWalk at[W];    // where each team's range begins
    Part part[2 * W];  // warp w's head slot (2w) and tail slot (2w + 1)
    Part beyond[2][kTeamMax];  // items that began before this block; items that go on behind it
    int32_t last[2 * kTeamMax];
  };
  static_assert(sizeof(Ctl) <= C::CTL, "control block");
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + W * C::WARP_BYTES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_wait();
  pdl_launch_dependents();

  // ---- the split: prefix sums of the rows' units --------------------------------
  // Up to 128 rows every warp sums them for itself (four rows per lane at most,
  // no barrier); more are shared among the block's threads.
  AttnWalk cw;  // where this warp stands
  int32_t u0, u1;            // units of this warp
  int32_t b0, share, rest, blocks;  // block c takes share units, one more when c < rest
  int32_t wshare, wrest;            // and so its teams
  int team, items, teams, my_team, member;  // items: of a team
  // false: this block has nothing to do.  A call of 2^31 units (16 TB of
  // keys and values and more) is refused: zeros.
  auto split = [&](int64_t rows_total) {
    items = p.c.kv_heads * p.head_groups;
    // teams leave more parts to join: not worth it for blocks with little work
    team = rows_total * items >= (int64_t)gridDim.x * kTeamUnits ? p.team : 1;
    items /= team;
    teams = W / team;
    my_team = warp / team;
    member = warp - my_team * team;
    if (rows_total > 0x7fffffffll / items) {
      if (tid == 0 && blockIdx.x == 0) flag_bad_index(p.status);
      uint4* out = static_cast<uint4*>(p.out);
      const int64_t n = (int64_t)p.m * p.q_heads * (D / 8);
      for (int64_t i = (int64_t)blockIdx.x * C::THREADS + tid; i < n; i += (int64_t)gridDim.x * C::THREADS)
        out[i] = make_uint4(0, 0, 0, 0);
      return false;
    }
    const int32_t total = (int32_t)rows_total * items, c = blockIdx.x;
    blocks = gridDim.x;
    if (total < blocks * p.min_units) blocks = (uint32_t)(total + p.min_units - 1) / (uint32_t)p.min_units;
    share = (uint32_t)total / (uint32_t)blocks;
    rest = total - share * blocks;
    b0 = c * share + (c < rest ? c : rest);
    const int32_t len = share + (c < rest ? 1 : 0);
    wshare = len / teams;
    wrest = len - wshare * teams;
    return c < blocks;
  };
  auto team_first = [&](int w) { return b0 + w * wshare + (w < wrest ? w : wrest); };
  // the block whose share holds unit u
  auto block_of = [&](int32_t u) {
    const uint32_t lead = (uint32_t)rest * (share + 1);
    return (uint32_t)u < lead ? (int32_t)((uint32_t)u / (uint32_t)(share + 1))
                              : rest + (int32_t)(((uint32_t)u - lead) / (uint32_t)share);
  };
  // the first tile at or after unit o of the row (it may be in the next row)
  auto place = [&](AttnWalk& w, int32_t o) {
    const int32_t unit = w.n + kItemCost;
    w.item = (uint32_t)o / (uint32_t)unit;
    w.j = o - w.item * unit - kItemCost;
    if (w.j < 0) w.j = 0;
  };
  if (tid < 2 * W) ctl->part[tid].n = 0;
  if (tid < 2 * kTeamMax) ctl->beyond[tid / kTeamMax][tid % kTeamMax].n = 0;
  if (p.m <= 128) {
    const int per = (p.m + 31) >> 5;
    AttnRow r[4];
    int32_t n[4];
    int64_t mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = lane * per + i;
      n[i] = 0;
      r[i] = {0, 0, 0};
      if (i < per && row < p.m) {
        bool bad;
        r[i] = attn_row(p, row, bad);
        if (bad && blockIdx.x == 0 && warp == 0) flag_bad_index(p.status);
        n[i] = r[i].tiles<TK>();
        mine += n[i] + kItemCost;
      }
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (!split(__shfl_sync(0xffffffffu, incl, 31))) return;
    u0 = team_first(my_team);
    u1 = team_first(my_team + 1);
    int32_t at = (int32_t)(incl - mine) * items;
    const int src = __ffs(__ballot_sync(0xffffffffu, u0 >= at && u0 < (int32_t)incl * items)) - 1;  // none when the range is empty
    const int sl = src < 0 ? 0 : src;
    AttnWalk w = {at, lane * per, 0, 0, n[0], r[0]};
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      at += (n[i - 1] ? n[i - 1] + kItemCost : 0) * items;
      if (n[i] && u0 >= at) w = {at, lane * per + i, 0, 0, n[i], r[i]};
    }
    cw.row = __shfl_sync(0xffffffffu, w.row, sl);
    cw.row_at = __shfl_sync(0xffffffffu, w.row_at, sl);
    cw.n = __shfl_sync(0xffffffffu, w.n, sl);
    cw.r.keys = __shfl_sync(0xffffffffu, w.r.keys, sl);
    cw.r.first = __shfl_sync(0xffffffffu, w.r.first, sl);
    cw.r.seq = __shfl_sync(0xffffffffu, w.r.seq, sl);
    place(cw, u0 - cw.row_at);
    __syncthreads();
  } else {
    const int per = (p.m + C::THREADS - 1) / C::THREADS;
    const int r0 = tid * per < p.m ? tid * per : p.m;
    const int r1 = r0 + per < p.m ? r0 + per : p.m;
    int64_t mine = 0;
    for (int i = r0; i < r1; ++i) {
      bool bad;
      mine += attn_row(p, i, bad).tiles<TK>() + kItemCost;
      if (bad && blockIdx.x == 0) flag_bad_index(p.status);
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) ctl->warp_sum[warp] = incl;
    __syncthreads();
    int64_t before = 0, rows_total = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < warp) before += ctl->warp_sum[i];
      rows_total += ctl->warp_sum[i];
    }
    if (!split(rows_total)) return;
    const int32_t b1 = team_first(teams);
    int32_t at = (int32_t)(before + incl - mine) * items;  // first unit of row r0
    if ((int32_t)(before + incl) * items > b0 && at < b1) {
      for (int i = r0; i < r1; ++i) {
        AttnWalk w;
        bool bad;
        w.r = attn_row(p, i, bad);
        w.n = w.r.tiles<TK>();
        w.row = i;
        w.row_at = at;
        at += (w.n + kItemCost) * items;
        for (int k = 0; k < teams; ++k) {
          const int32_t s = team_first(k);
          if (s >= w.row_at && s < at) {
            place(w, s - w.row_at);
            ctl->at[k] = w;
          }
        }
      }
    }
    __syncthreads();
    u0 = team_first(my_team);
    u1 = team_first(my_team + 1);
    if (u0 < u1) cw = ctl->at[my_team];
  }
  // unit of the tile that a walk stands at
  auto unit_of = [&](const AttnWalk& w) { return w.row_at + w.item * (w.n + kItemCost) + kItemCost + w.j; };

  uint8_t* ring = smem + warp * C::WARP_BYTES;
  float* head_slot = reinterpret_cast<float*>(ring + C::RING);  // O of the first item when it began before the warp
  float* tail_slot = reinterpret_cast<float*>(ring);            // O of the last item when it goes on (ring drained)
  const uint32_t ring_u = smem_u32(ring);

  if (u0 < u1 && unit_of(cw) < u1) {
    AttnWalk pw = cw;  // producer: the tile whose pages are looked up next
    bool more = true;  // pw stands at a tile of this warp

    // look-up state of the producer: lane l < TK holds key l of the tile
    constexpr uint32_t FULL_MASK = 0xffffffffu >> (32 - TK);
    struct Look {
      int32_t page;
      uint32_t off;  // offset inside the page, head included
      bool valid;
    };
    auto look = [&]() {
      Look l = {-1, 0u, false};
      if (more) {
        const int32_t idx = pw.j * TK + (lane & (TK - 1));
        if (idx < pw.r.keys) {
          const uint32_t t = (uint32_t)(pw.r.first + idx);
          const uint32_t pi = (__umulhi(t, p.page_mul) + t) >> p.page_shift;
          l.page = p.c.pages[(int64_t)pw.r.seq * p.c.max_pages + pi];
          l.off = (t - pi * (uint32_t)p.c.page_size) * p.token_step +
                  (uint32_t)((pw.item * team + member) / p.head_groups) * p.head_step;
          l.valid = true;
        }
        attn_next<TK>(p, pw, items);
        more = pw.row < p.m && unit_of(pw) < u1;
      }
      return l;
    };
    // a lane copies chunk lane % CPR of every (32 / CPR)-th key (rows of 12 and 6 chunks: any chunk)
    constexpr bool EVEN = 32 % C::CPR == 0;
    uint64_t masks = 0;  // valid keys of the tiles in flight, TK bits each, the oldest highest
    int stage_in = 0;
    auto copy = [&](const Look& l) {  // start the copies of a looked-up tile
      const bool ok = l.valid && l.page >= 0 && l.page < p.c.n_pages;
      if (l.valid && !ok) flag_bad_index(p.status);
      const uint32_t o = ok ? (uint32_t)l.page * p.page_step + l.off : 0u;
      const uint32_t vm = __ballot_sync(0xffffffffu, ok) & FULL_MASK;
      masks = (masks << TK) | vm;
      if (vm) {
        const uint32_t base = ring_u + stage_in * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::CPR * TK / 32; ++i) {
          const int c = i * 32 + lane;
          const int r = EVEN ? i * (32 / C::CPR) + lane / C::CPR : c / C::CPR;
          const int ch = EVEN ? lane % C::CPR : c - r * C::CPR;
          const uint64_t bo = (uint64_t)__shfl_sync(0xffffffffu, o, r) * p.unit + ch * 16;
          const uint32_t d = base + r * C::RB + (ch ^ C::swz(r)) * 16;
          const bool in = vm == FULL_MASK || (vm >> r & 1);
          cp_async16(d, static_cast<const uint8_t*>(p.c.k) + bo, in);
          cp_async16(d + TK * C::RB, static_cast<const uint8_t*>(p.c.v) + bo, in);
        }
      }
      cp_async_commit();
      if (++stage_in == S) stage_in = 0;
    };

    Look next;
    {
      Look l[S - 1];  // the first look-ups together: their latencies overlap
#pragma unroll
      for (int i = 0; i < S - 1; ++i) l[i] = look();
      next = look();
#pragma unroll
      for (int i = 0; i < S - 1; ++i) copy(l[i]);
    }

    uint32_t qf[NT][MT][2];
    float o[MT][NT][4];
    float mx[NT][2], sum[NT][2];
    float sc = 0.f, vscale = 1.f;
    bool fresh = true;       // load the item's queries before the next tile
    bool began_before = cw.j > 0;
    int stage_out = 0;

    // this lane's query column and the address of its fragment elements
    auto head_of = [&](int item, int col) {  // query head of a column, or -1
      const int kvh = item / p.head_groups, hg = item - kvh * p.head_groups;
      const int g = hg * COLS + col;
      return g < p.group ? kvh * p.group + g : -1;
    };

    for (bool done = false; !done;) {
      if (fresh) {
        fresh = false;
        const int item = cw.item * team + member, kvh = item / p.head_groups;
        sc = p.scale * 1.44269504088896340736f * (p.c.ks ? p.c.ks[kvh] : 1.f);
        // a negative scale turns the queries around, so that the largest product has the largest score
        const uint32_t flip = sc < 0.f ? 0x80008000u : 0u;
        sc = fabsf(sc);
        vscale = p.c.vs ? p.c.vs[kvh] : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int h = head_of(item, nt * 8 + (lane >> 2));
          const uint16_t* qp = static_cast<const uint16_t*>(p.q) + ((int64_t)cw.row * p.q_heads + (h < 0 ? 0 : h)) * D;
#pragma unroll
          for (int ks = 0; ks < MT; ++ks) {
            uint32_t x0 = 0, x1 = 0;
            if (h >= 0) {
              if constexpr (F8) {  // k slots 2q.. and 2q+8.. of a step hold features 4q.. and 4q+2..
                const uint2 v = *reinterpret_cast<const uint2*>(qp + ks * 16 + (lane & 3) * 4);
                x0 = v.x;
                x1 = v.y;
              } else {
                x0 = *reinterpret_cast<const uint32_t*>(qp + ks * 16 + (lane & 3) * 2);
                x1 = *reinterpret_cast<const uint32_t*>(qp + ks * 16 + 8 + (lane & 3) * 2);
              }
            }
            qf[nt][ks][0] = x0 ^ flip;
            qf[nt][ks][1] = x1 ^ flip;
          }
          mx[nt][0] = mx[nt][1] = -INFINITY;
          sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
        }
      }

      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t vm = (uint32_t)(masks >> (TK * (S - 2))) & (0xffffffffu >> (32 - TK));
      copy(next);  // into the stage that the previous tile has left
      next = look();

      if (vm) {
        const uint32_t kb = ring_u + stage_out * C::STAGE;
        const uint32_t vb = kb + TK * C::RB;
        // S^T, in two independent sums per 16 keys
        float s[KT][NT][4], s2[KT][NT][4];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[kt][nt][i] = s2[kt][nt][i] = 0.f;
        // this lane's row of the 8x8 matrices, and its chunk: ((step, half) ^ swz(row)) * 16
        const int krow = (lane & 7) + ((lane >> 3) & 1) * 8;
        const uint32_t ka = kb + krow * C::RB;
        const uint32_t kx = ((lane >> 4) ^ C::swz(krow)) * 16;
        if constexpr (!F8) {
#pragma unroll
          for (int ks = 0; ks < MT; ++ks)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              uint32_t a[4];
              ldsm4(a, ka + kt * 16 * C::RB + (kx ^ (ks * 32)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16<BF>((ks & 1) ? s2[kt][nt] : s[kt][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
            }
        } else {
#pragma unroll
          for (int ks = 0; ks < MT; ks += 2)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              uint32_t r[4];
              ldsm4(r, ka + kt * 16 * C::RB + (kx ^ (ks * 16)));
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t a[4];
                e4m3x4_to_h2(r[2 * u], a[0], a[2]);
                e4m3x4_to_h2(r[2 * u + 1], a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16<BF>(u ? s2[kt][nt] : s[kt][nt], a, qf[nt][ks + u][0], qf[nt][ks + u][1]);
              }
            }
        }
        // softmax: lane holds keys lane/4 and lane/4 + 8 (of each 16) of heads
        // 2(lane%4) and +1; mx is the largest product, weights 2^(sc (x - mx))
        float tm[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tm[nt][i] = -INFINITY;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int r = 0; r < 2; ++r) s[kt][nt][2 * r + i] += s2[kt][nt][2 * r + i];
          }
        if (vm != FULL_MASK) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const bool in = (vm >> (kt * 16 + r * 8 + (lane >> 2))) & 1;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  if (!in) s[kt][nt][2 * r + i] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int r = 0; r < 2; ++r) tm[nt][i] = fmaxf(tm[nt][i], s[kt][nt][2 * r + i]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) tm[nt][i] = fmaxf(tm[nt][i], __shfl_xor_sync(0xffffffffu, tm[nt][i], d));
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) up |= tm[nt][i] > mx[nt][i];
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float mn = fmaxf(mx[nt][i], tm[nt][i]);
              const float f = mx[nt][i] == -INFINITY ? 0.f : ex2((mx[nt][i] - mn) * sc);
              mx[nt][i] = mn;
              sum[nt][i] *= f;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                o[mt][nt][i] *= f;
                o[mt][nt][i + 2] *= f;
              }
            }
        }
        // P^T as the B operand, in terms that keep binary32 accuracy (AttnWeights)
        uint32_t pt[TERMS][KT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float m0[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) m0[i] = mx[nt][i] == -INFINITY ? 0.f : AttnWeights<T>::UP - mx[nt][i] * sc;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float e[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float x = s[kt][nt][2 * r + i];
                // x is -inf for hidden keys (and sc may be 0)
                e[i] = vm == FULL_MASK || x != -INFINITY ? ex2(fmaf(x, sc, m0[i])) : 0.f;
                sum[nt][i] += e[i];
              }
              uint32_t t[TERMS];
              AttnWeights<T>::split(e[0], e[1], t);
#pragma unroll
              for (int k = 0; k < TERMS; ++k) pt[k][kt][nt][r] = transpose8(t[k]);
            }
        }
        // O^T: the tile's share, two row tiles at a time, is added to O by the
        // threads.  The tensor core drops the bits below its accumulator's last
        // place, which in one chain over 2^20 keys made outputs 1% too small.
        // Small terms first, so that most of them are added to small sums.
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2) {
          float t[2][NT][4];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) t[u][nt][i] = 0.f;
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            uint32_t a[2][4];
            if constexpr (!F8) {
              const int vrow = (lane & 7) + (lane >> 4) * 8;
              const uint32_t va = vb + (kt * 16 + vrow) * C::RB;
              const uint32_t vx = (((lane >> 3) & 1) ^ C::swz(vrow)) * 16;
              ldsm4_t(a[0], va + (vx ^ (mt * 32)));
              ldsm4_t(a[1], va + (vx ^ (mt * 32 + 32)));
            } else {
              // a 16-bit element of the transposed load is a pair of neighbouring
              // features: MMA rows r and r + 8 are features 2r and 2r + 1
              uint32_t r[4];
              ldsm4_t(r, vb + (kt * 16 + krow) * C::RB + (kx ^ (mt * 16)));
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                e4m3x4_to_h2(__byte_perm(r[2 * u], 0, 0x3120), a[u][0], a[u][1]);
                e4m3x4_to_h2(__byte_perm(r[2 * u + 1], 0, 0x3120), a[u][2], a[u][3]);
              }
            }
#pragma unroll
            for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma16<BF>(t[u][nt], a[u], pt[k][kt][nt][0], pt[k][kt][nt][1]);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[mt + u][nt][i] += t[u][nt][i];
        }
      }
      if (++stage_out == S) stage_out = 0;
      __syncwarp();

      // ---- end of the item or of the warp's range ---------------------------------
      const AttnWalk tile = cw;
      const bool item_end = cw.j + 1 == cw.n;
      attn_next<TK>(p, cw, items);
      done = cw.row >= p.m || unit_of(cw) >= u1;
      if (item_end || done) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) sum[nt][i] += __shfl_xor_sync(0xffffffffu, sum[nt][i], d);
        if (item_end && !began_before) {
          // whole item: normalise, round, transpose to [head][feature], write
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float inv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) inv[i] = sum[nt][i] == 0.f ? 0.f : vscale / sum[nt][i];
            const int h = head_of(tile.item * team + member, nt * 8 + (lane >> 2));
            uint16_t* op = static_cast<uint16_t*>(p.out) + ((int64_t)tile.row * p.q_heads + (h < 0 ? 0 : h)) * D;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const float* v = o[mt][nt];
              const float y0 = v[0] * inv[0], y1 = v[1] * inv[1], y2 = v[2] * inv[0], y3 = v[3] * inv[1];
              const uint32_t t0 = transpose8(p.out_bf16 ? KvElem<KV_BF16>::pack2(y0, y1) : f2_to_h2(y0, y1));
              const uint32_t t1 = transpose8(p.out_bf16 ? KvElem<KV_BF16>::pack2(y2, y3) : f2_to_h2(y2, y3));
              if (h >= 0) {
                if constexpr (F8) {  // t0: features 4q, 4q+2; t1: 4q+1, 4q+3
                  *reinterpret_cast<uint2*>(op + mt * 16 + (lane & 3) * 4) =
                      make_uint2(__byte_perm(t0, t1, 0x5410), __byte_perm(t0, t1, 0x7632));
                } else {
                  *reinterpret_cast<uint32_t*>(op + mt * 16 + (lane & 3) * 2) = t0;
                  *reinterpret_cast<uint32_t*>(op + mt * 16 + 8 + (lane & 3) * 2) = t1;
                }
              }
            }
          }
        } else {
          if (!item_end) {
            cp_async_wait<0>();  // the ring is empty before its bytes are reused
            __syncwarp();
          }
          float* dst = item_end ? head_slot : tail_slot;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int d0 = F8 ? mt * 16 + 2 * (lane >> 2) : mt * 16 + (lane >> 2);
            const int d1 = F8 ? d0 + 1 : d0 + 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int col = nt * 8 + (lane & 3) * 2;
              *reinterpret_cast<float2*>(dst + d0 * COLS + col) = make_float2(o[mt][nt][0], o[mt][nt][1]);
              *reinterpret_cast<float2*>(dst + d1 * COLS + col) = make_float2(o[mt][nt][2], o[mt][nt][3]);
            }
          }
          if (lane < 4) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int col = nt * 8 + lane * 2 + i;
                dst[D * COLS + col] = mx[nt][i] == -INFINITY ? -INFINITY : mx[nt][i] * sc;
                dst[D * COLS + COLS + col] = sum[nt][i];
              }
          }
          if (lane == 0)
            ctl->part[2 * warp + (item_end ? 0 : 1)] = {tile.row_at + tile.item * (tile.n + kItemCost) + kItemCost, tile.n,
                                                        tile.row, tile.item * team + member, member};
        }
        began_before = false;
        fresh = true;
      }
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  // ---- join (see AttnSum) -----------------------------------------------------------
  const int32_t b1 = team_first(teams);
  uint32_t live, same;  // slots with parts; of these, the ones of the same item
  {
    int32_t id = -1 - lane;
    if (lane < 2 * W && ctl->part[lane].n) id = ctl->part[lane].row * items * team + ctl->part[lane].item;
    live = __ballot_sync(0xffffffffu, id >= 0);
    same = __match_any_sync(0xffffffffu, id);
  }
  AttnSum<D, COLS, C::THREADS> sum;
  // part of an item in block c: the second set of slots if the item begins there
  auto global = [&](int c, bool second, int mem) {
    return p.partials + (((int64_t)c * 2 + second) * kTeamMax + mem) * C::PART;
  };
  bool any = false;
  while (live) {  // the same in all warps
    const int k0 = __ffs(live) - 1;
    uint32_t parts = __shfl_sync(0xffffffffu, same, k0);
    live &= ~parts;
    const Part g = ctl->part[k0];
    sum.clear();
#pragma unroll 1
    while (parts) {
      const int ka = __ffs(parts) - 1;
      parts &= parts - 1;
      const int kb = parts ? __ffs(parts) - 1 : ka;
      const int n = parts ? 2 : 1;
      parts &= parts - 1;
      sum.template add<2>(n, [&](int i) {
        const int k = i ? kb : ka;
        return reinterpret_cast<const float*>(smem + (k >> 1) * C::WARP_BYTES + ((k & 1) ? 0 : C::RING));
      });
    }
    if (g.first >= b0 && g.first + g.n <= b1) {
      sum.write(p, g.row, g.item);
    } else {
      any = true;
      const bool second = g.first >= b0;
      sum.store(global(blockIdx.x, second, g.member));
      if (tid == 0) ctl->beyond[second][g.member] = g;
    }
  }
  if (!any) return;
  __syncthreads();
  auto arrive = [&](int32_t* counter, int n) {  // in one thread: true for the last of n
    const int32_t old = atomicAdd(counter, 1);
    if (old == n - 1) *counter = 0;
    return old == n - 1;
  };
  // the blocks of an item: ca .. ca + n - 1
  auto extent = [&](const Part& g, int& ca, int& n) {
    ca = block_of(g.first);
    n = block_of(g.first + g.n - 1) - ca + 1;
    return ((int)blockIdx.x - ca) / kJoin * kJoin;  // first of this block's group
  };
  if (tid < 2 * kTeamMax) {
    const Part g = ctl->beyond[tid / kTeamMax][tid % kTeamMax];
    ctl->last[tid] = 0;
    if (g.n) {
      int ca, n;
      const int i0 = extent(g, ca, n);
      __threadfence();
      ctl->last[tid] = arrive(p.counters + (2 * (ca + i0) + (i0 == 0)) * kTeamMax + g.member, n - i0 < kJoin ? n - i0 : kJoin);
      __threadfence();
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int s = 0; s < 2 * kTeamMax; ++s) {
    if (!ctl->last[s]) continue;  // the same in all threads
    const Part g = ctl->beyond[s / kTeamMax][s % kTeamMax];
    int ca, n;
    const int i0 = extent(g, ca, n);
    sum.sum(n - i0 < kJoin ? n - i0 : kJoin, [&](int i) { return global(ca + i0 + i, i0 + i == 0, g.member); });
    if (n > kJoin) {
      __syncthreads();  // every thread has read the group's parts, of which the first is replaced
      sum.store(global(ca + i0, i0 == 0, g.member));
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        ctl->last[s] = arrive(p.counters + kTopCounters + ca * kTeamMax + g.member, (n + kJoin - 1) / kJoin);
        __threadfence();
      }
      __syncthreads();
      if (!ctl->last[s]) continue;
      sum.sum((n + kJoin - 1) / kJoin, [&](int i) { return global(ca + i * kJoin, i == 0, g.member); });
    }
    sum.write(p, g.row, g.item);
  }
}

}  // namespace tq
