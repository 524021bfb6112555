// tq_serve.cu -- the C ABI's paged cache, attention and adapter entry points
// (see include/tq.h): argument checks and launches.  No allocation, no
// synchronisation.
#include <math.h>
#include <string.h>

#include "../../include/tq.h"
#include "tq_attn.cuh"
#include "tq_host.cuh"
#include "tq_kv.cuh"
#include "tq_lora.cuh"

using namespace tq_host;

namespace {

constexpr int32_t kMaxM = 4096;  // tokens per call, as in tq_gemm

int32_t* status_word(void* ws) { return reinterpret_cast<int32_t*>(static_cast<char*>(ws) + TQ_STATUS_OFFSET); }

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_cache(const tq_kv_cache_t* c) {
  if (!c) return TQ_ERR_NULL;
  if (c->dtype != TQ_F16 && c->dtype != TQ_BF16 && c->dtype != TQ_E4M3) return TQ_ERR_VALUE;
  if (c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128 && c->head_dim != 256) return TQ_ERR_SHAPE;
  if (c->n_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->n_seqs < 1 || c->max_pages < 1) return TQ_ERR_SHAPE;
  if ((int64_t)c->page_size * c->max_pages > 0x7fffffff) return TQ_ERR_SHAPE;
  if (!c->k_d || !c->v_d || !c->pages_d) return TQ_ERR_NULL;
  const int64_t eb = c->dtype == TQ_E4M3 ? 1 : 2;
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return TQ_ERR_VALUE;
  if ((c->page_stride * eb) % 16 || (c->token_stride * eb) % 16 || (c->head_stride * eb) % 16) return TQ_ERR_ALIGN;
  if (!aligned16(c->k_d) || !aligned16(c->v_d) || !aligned_to(c->pages_d, 4) || !aligned_to(c->k_scale_d, 4) ||
      !aligned_to(c->v_scale_d, 4))
    return TQ_ERR_ALIGN;
  if (c->dtype != TQ_E4M3 && (c->k_scale_d || c->v_scale_d)) return TQ_ERR_VALUE;
  return TQ_OK;
}

tq::KvView cache_view(const tq_kv_cache_t* c) {
  tq::KvView v;
  v.k = c->k_d;
  v.v = c->v_d;
  v.pages = c->pages_d;
  v.ks = c->k_scale_d;
  v.vs = c->v_scale_d;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.kv_heads = c->kv_heads;
  v.head_dim = c->head_dim;
  v.n_seqs = c->n_seqs;
  v.max_pages = c->max_pages;
  return v;
}

int check_heads(const tq_kv_cache_t* c, int32_t m, int32_t q_heads) {
  if (m < 0 || m > kMaxM) return TQ_ERR_SHAPE;
  if (q_heads < 1 || q_heads % c->kv_heads != 0) return TQ_ERR_SHAPE;
  if ((int64_t)(q_heads + 2 * (int64_t)c->kv_heads) * c->head_dim > 1 << 24) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return TQ_ERR_WORKSPACE;
  if (!aligned16(ws)) return TQ_ERR_ALIGN;
  return TQ_OK;
}

// Attention: one block per SM; two partial results per block.
constexpr int kAttnMaxBlocks = 148;
constexpr int kAttnMinUnits = 6;   // tiles (and item costs) a block takes before another is used

int attn_cols(const tq_kv_cache_t* c, int32_t q_heads) { return q_heads / c->kv_heads <= 8 ? 8 : 16; }

size_t attn_ws_bytes(const tq_kv_cache_t* c, int32_t q_heads) {
  const int cols = attn_cols(c, q_heads);
  return kCounterBytes + (size_t)kAttnMaxBlocks * 2 * tq::kTeamMax * (c->head_dim * cols + 2 * cols) * sizeof(float);
}

// Multiplier and shift of an exact division of values below 2^31 by d:
// n / d = (umulhi(n, mul) + n) >> shift (Granlund and Montgomery 1994).
void divider(uint32_t d, uint32_t* mul, uint32_t* shift) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  *mul = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  *shift = l;
}

// The cache's strides as 32-bit multiples of the largest power of two (4 KB at
// most) that divides them; false when its last element is beyond 32 bits of them.
bool attn_steps(const tq_kv_cache_t* c, tq::AttnParams* p) {
  const int64_t eb = c->dtype == TQ_E4M3 ? 1 : 2;
  const int64_t ps = c->page_stride * eb, ts = c->token_stride * eb, hs = c->head_stride * eb;
  int64_t unit = 4096;
  while ((ps | ts | hs) & (unit - 1)) unit >>= 1;
  // products of the sizes with the strides, in units, checked without overflow
  const double last = ((double)(c->n_pages - 1) * (double)ps + (double)(c->page_size - 1) * (double)ts +
                       (double)(c->kv_heads - 1) * (double)hs) / (double)unit;
  if (last > 4294967295.0 || ps / unit > 0xffffffffll || ts / unit > 0xffffffffll || hs / unit > 0xffffffffll) return false;
  p->unit = (uint32_t)unit;
  p->page_step = (uint32_t)(ps / unit);
  p->token_step = (uint32_t)(ts / unit);
  p->head_step = (uint32_t)(hs / unit);
  return true;
}

// Warps that work together on neighbouring items (tq_attn.cuh): enough that
// their keys make 256 bytes in a row, or that all query heads of a key head are
// among them; a power of two that divides the items and the block's warps.
int attn_team(const tq_kv_cache_t* c, int head_groups, int warps) {
  const int row = c->head_dim * (c->dtype == TQ_E4M3 ? 1 : 2);
  int want = 1;
  while (want < head_groups) want *= 2;
  if (c->head_stride == c->head_dim && c->page_size > 1)
    while (want * row < 256) want *= 2;
  int team = 1;
  while (2 * team <= want && 2 * team <= tq::kTeamMax && (c->kv_heads * head_groups) % (2 * team) == 0 &&
         warps % (2 * team) == 0)
    team *= 2;
  return team;
}

template <int T, int D, int NT>
int attn_launch(tq::AttnParams p, const tq_kv_cache_t* c, int sms, cudaStream_t stream) {
  using C = tq::AttnCfg<T, D, NT>;
  auto kern = tq::attn_kernel<T, D, NT>;
  static int configured[kMaxDevices];
  int dev = 0;
  TQ_CUDA(cudaGetDevice(&dev));
  if (!configured[dev]) {
    TQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
    configured[dev] = 1;
  }
  p.team = attn_team(c, p.head_groups, C::WARPS);
  const int grid = sms < kAttnMaxBlocks ? sms : kAttnMaxBlocks;
  return launch(kern, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, stream, p);
}

template <int T, int D>
int attn_launch_d(const tq::AttnParams& p, const tq_kv_cache_t* c, int cols, int sms, cudaStream_t stream) {
  return cols == 8 ? attn_launch<T, D, 1>(p, c, sms, stream) : attn_launch<T, D, 2>(p, c, sms, stream);
}

template <int T>
int attn_launch_t(const tq::AttnParams& p, const tq_kv_cache_t* c, int cols, int sms, cudaStream_t stream) {
  switch (p.c.head_dim) {
    case 64: return attn_launch_d<T, 64>(p, c, cols, sms, stream);
    case 96: return attn_launch_d<T, 96>(p, c, cols, sms, stream);
    case 128: return attn_launch_d<T, 128>(p, c, cols, sms, stream);
    default: return attn_launch_d<T, 256>(p, c, cols, sms, stream);
  }
}

int check_lora(const tq_lora_t* l) {
  if (!l) return TQ_ERR_NULL;
  if (l->dtype != TQ_F16 && l->dtype != TQ_BF16) return TQ_ERR_VALUE;
  if (l->n_adapters < 1 || l->n_adapters > TQ_LORA_MAX_ADAPTERS || l->n < 1 || l->k < 512 || l->k % 512 != 0) return TQ_ERR_SHAPE;
  if (l->rank < 8 || l->rank > TQ_LORA_MAX_RANK || l->rank % 8 != 0) return TQ_ERR_SHAPE;
  if (!l->a_d || !l->b_d) return TQ_ERR_NULL;
  if (!aligned16(l->a_d) || !aligned16(l->b_d) || !aligned_to(l->scale_d, 4)) return TQ_ERR_ALIGN;
  return TQ_OK;
}

// Splits of k for more than kLoraInBlock tokens: about one (tile, split) pair
// for each of two blocks per SM, and 512 features of x for each at least.
int lora_splits(const tq_lora_t* l, int32_t m) {
  int s = 2 * kAttnMaxBlocks / ((m + tq::kLoraTile - 1) / tq::kLoraTile);
  if (s > 8) s = 8;
  if (s > l->k / 512) s = l->k / 512;
  return s < 1 ? 1 : s;
}

constexpr size_t kLoraPlanBytes = (tq::kPlanInts * sizeof(int32_t) + 255) / 256 * 256;

// Workspace of more than kLoraInBlock tokens: [counters][plan][A x of each
// split][its terms][multipliers]
size_t lora_terms_off(const tq_lora_t* l, int32_t m) {
  return kCounterBytes + kLoraPlanBytes + ((size_t)lora_splits(l, m) * m * l->rank * sizeof(float) + 255) / 256 * 256;
}
size_t lora_mul_off(const tq_lora_t* l, int32_t m) {
  return lora_terms_off(l, m) + ((size_t)m * 3 * l->rank * sizeof(uint16_t) + 255) / 256 * 256;
}

size_t lora_ws_bytes(const tq_lora_t* l, int32_t m) {
  if (m <= tq::kLoraInBlock) return kCounterBytes;
  return lora_mul_off(l, m) + (size_t)m * sizeof(float);
}

// What the query answers: enough for every call of up to m tokens.  (Fewer
// tokens can need more, since they take more splits; within a number of tiles
// the need grows with m.)
size_t lora_ws_query(const tq_lora_t* l, int32_t m) {
  size_t most = lora_ws_bytes(l, m);
  for (int32_t t = m / tq::kLoraTile * tq::kLoraTile; t > tq::kLoraInBlock; t -= tq::kLoraTile) {
    const size_t b = lora_ws_bytes(l, t);
    if (b > most) most = b;
  }
  return most;
}

template <bool BF16, int PANELS>
int lora_expand_launch(const tq::LoraParams& p, int sms, int64_t units, cudaStream_t stream) {
  auto kern = tq::lora_expand_kernel<BF16, PANELS>;
  constexpr size_t smem = sizeof(tq::LoraSmem<PANELS>) + 1024;
  static int configured[kMaxDevices];
  int dev = 0;
  TQ_CUDA(cudaGetDevice(&dev));
  if (!configured[dev]) {
    TQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    configured[dev] = 1;
  }
  int64_t grid = (int64_t)sms * (PANELS == 1 ? 3 : 2);
  if (grid > units) grid = units;
  return launch(kern, dim3((unsigned)grid), dim3(tq::LORA_THREADS), smem, stream, p);
}

template <bool BF16>
int lora_prompt(const tq::LoraParams& p, int sms, int64_t tiles, cudaStream_t stream) {
  int st = launch(tq::lora_plan_kernel, dim3(1), dim3(1024), 0, stream, p);
  if (st != TQ_OK) return st;
  int64_t grid = (int64_t)sms * 2;
  if (grid > tiles * p.splits) grid = tiles * p.splits;
  st = launch(tq::lora_shrink_kernel<BF16>, dim3((unsigned)grid), dim3(tq::LORA_THREADS), 0, stream, p);
  if (st != TQ_OK) return st;
  const int64_t units = tiles * ((p.n + 127) / 128);
  return p.rank <= 64 ? lora_expand_launch<BF16, 1>(p, sms, units, stream)
                      : lora_expand_launch<BF16, 2>(p, sms, units, stream);
}

}  // namespace

extern "C" {

int tq_kv_append_workspace(size_t* bytes) {
  if (!bytes) return TQ_ERR_NULL;
  *bytes = kCounterBytes;
  return TQ_OK;
}

int tq_kv_append(const tq_kv_cache_t* cache, const float* qkv_d, int64_t qkv_stride, int32_t m, int32_t q_heads,
                 const int32_t* seq_d, const int32_t* pos_d, const double* freq_d, int32_t rot_dim,
                 int32_t interleaved, void* q_out_d, void* workspace_d, size_t ws_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != TQ_OK) return st;
  st = check_heads(cache, m, q_heads);
  if (st != TQ_OK) return st;
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16 != 0) return TQ_ERR_SHAPE;
  if (interleaved != 0 && interleaved != 1) return TQ_ERR_VALUE;
  if (qkv_stride < (int64_t)(q_heads + 2 * cache->kv_heads) * cache->head_dim) return TQ_ERR_SHAPE;
  if (m == 0) return TQ_OK;
  if (!qkv_d || !pos_d || !q_out_d || (rot_dim > 0 && !freq_d)) return TQ_ERR_NULL;
  if (!aligned16(qkv_d) || qkv_stride % 4 != 0 || !aligned16(q_out_d) || !aligned_to(pos_d, 4) ||
      !aligned_to(seq_d, 4) || !aligned_to(freq_d, 8))
    return TQ_ERR_ALIGN;
  st = check_ws(workspace_d, ws_bytes, kCounterBytes);
  if (st != TQ_OK) return st;
  int sms = 0;
  st = check_arch(&sms);
  if (st != TQ_OK) return st;
  tq::AppendParams p;
  p.c = cache_view(cache);
  p.qkv = qkv_d;
  p.qkv_stride = qkv_stride;
  p.q_out = q_out_d;
  p.seq = seq_d;
  p.pos = pos_d;
  p.freq = freq_d;
  p.m = m;
  p.q_heads = q_heads;
  p.rot = rot_dim;
  p.interleaved = interleaved;
  p.status = status_word(workspace_d);
  const int units = (q_heads + 2 * cache->kv_heads) * (cache->head_dim / 16);
  // many tokens: whole tokens to as many blocks as run at once; few: their heads are spread over blocks.
  // Whole against spread (32/8 heads x 128, fp16): 32 tokens 3.6 against 2.7 us, 256 4.4 and 4.5, 518 6.2 and 6.6,
  // 2000 16.2 against 18.5; e4m3: 32 tokens 5.0 against 3.9, 400 8.2 and 7.6, 700 8.5 against 10.0, 2000 19.5 against 23.3
  const int32_t at_once = sms * tq::append_blocks(cache->dtype);
  const bool many = m >= at_once / 2;
  const int parts = many ? 1 : (units + tq::AP_THREADS - 1) / tq::AP_THREADS;
  const dim3 grid((unsigned)(m < at_once ? m : at_once), (unsigned)parts), block(tq::AP_THREADS);
  cudaStream_t s = (cudaStream_t)stream;
  switch (cache->dtype) {
    case TQ_F16: return launch(tq::append_kernel<tq::KV_F16>, grid, block, 0, s, p);
    case TQ_BF16: return launch(tq::append_kernel<tq::KV_BF16>, grid, block, 0, s, p);
    default: return launch(tq::append_kernel<tq::KV_E4M3>, grid, block, 0, s, p);
  }
}

int tq_attn_workspace(const tq_kv_cache_t* cache, int32_t m, int32_t q_heads, size_t* bytes) {
  if (!bytes) return TQ_ERR_NULL;
  int st = check_cache(cache);
  if (st != TQ_OK) return st;
  st = check_heads(cache, m, q_heads);
  if (st != TQ_OK) return st;
  *bytes = attn_ws_bytes(cache, q_heads);
  return TQ_OK;
}

int tq_attn(const tq_kv_cache_t* cache, const void* q_d, int32_t m, int32_t q_heads, const int32_t* seq_d,
            const int32_t* pos_d, float scale, int32_t window, void* out_d, int32_t out_dtype, void* workspace_d,
            size_t ws_bytes, void* stream) {
  int st = check_cache(cache);
  if (st != TQ_OK) return st;
  st = check_heads(cache, m, q_heads);
  if (st != TQ_OK) return st;
  if (out_dtype != TQ_F16 && out_dtype != TQ_BF16) return TQ_ERR_VALUE;
  if (!isfinite(scale) || window < 0) return TQ_ERR_VALUE;
  tq::AttnParams p;
  if (!attn_steps(cache, &p)) return TQ_ERR_SHAPE;
  if (m == 0) return TQ_OK;
  if (!q_d || !pos_d || !out_d) return TQ_ERR_NULL;
  if (!aligned16(q_d) || !aligned16(out_d) || !aligned_to(pos_d, 4) || !aligned_to(seq_d, 4)) return TQ_ERR_ALIGN;
  st = check_ws(workspace_d, ws_bytes, attn_ws_bytes(cache, q_heads));
  if (st != TQ_OK) return st;
  int sms = 0;
  st = check_arch(&sms);
  if (st != TQ_OK) return st;
  p.c = cache_view(cache);
  p.q = q_d;
  p.seq = seq_d;
  p.pos = pos_d;
  p.out = out_d;
  p.m = m;
  p.q_heads = q_heads;
  p.window = window;
  p.scale = scale;
  p.group = q_heads / cache->kv_heads;
  const int cols = attn_cols(cache, q_heads);
  p.head_groups = (p.group + cols - 1) / cols;
  p.min_units = kAttnMinUnits;
  divider((uint32_t)cache->page_size, &p.page_mul, &p.page_shift);
  p.out_bf16 = out_dtype == TQ_BF16;
  p.counters = static_cast<int32_t*>(workspace_d);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace_d) + kCounterBytes);
  p.status = status_word(workspace_d);
  cudaStream_t s = (cudaStream_t)stream;
  switch (cache->dtype) {
    case TQ_F16: return attn_launch_t<tq::KV_F16>(p, cache, cols, sms, s);
    case TQ_BF16: return attn_launch_t<tq::KV_BF16>(p, cache, cols, sms, s);
    default: return attn_launch_t<tq::KV_E4M3>(p, cache, cols, sms, s);
  }
}

int tq_lora_workspace(const tq_lora_t* lora, int32_t m, size_t* bytes) {
  if (!bytes) return TQ_ERR_NULL;
  int st = check_lora(lora);
  if (st != TQ_OK) return st;
  if (m < 0 || m > kMaxM) return TQ_ERR_SHAPE;
  *bytes = lora_ws_query(lora, m);
  return TQ_OK;
}

int tq_lora(const tq_lora_t* lora, const void* x_d, int32_t m, const int32_t* adapter_d, const float* y_d,
            int64_t y_stride, float* out_d, int64_t out_stride, void* workspace_d, size_t ws_bytes, void* stream) {
  int st = check_lora(lora);
  if (st != TQ_OK) return st;
  if (m < 0 || m > kMaxM || y_stride < lora->n || out_stride < lora->n) return TQ_ERR_SHAPE;
  if (y_stride > (1 << 20) || out_stride > (1 << 20)) return TQ_ERR_SHAPE;  // m rows stay inside 32-bit offsets
  if (m > 1 && out_d == y_d && out_stride != y_stride) return TQ_ERR_SHAPE;  // rows would be overwritten before they are read
  if (m == 0) return TQ_OK;
  if (!x_d || !adapter_d || !y_d || !out_d) return TQ_ERR_NULL;
  if (!aligned16(x_d) || !aligned_to(adapter_d, 4) || !aligned_to(y_d, 4) || !aligned_to(out_d, 4)) return TQ_ERR_ALIGN;
  st = check_ws(workspace_d, ws_bytes, lora_ws_bytes(lora, m));
  if (st != TQ_OK) return st;
  int sms = 0;
  st = check_arch(&sms);
  if (st != TQ_OK) return st;
  tq::LoraParams p;
  p.a = lora->a_d;
  p.b = lora->b_d;
  p.scale = lora->scale_d;
  p.x = x_d;
  p.adapter = adapter_d;
  p.y = y_d;
  p.out = out_d;
  p.y_stride = y_stride;
  p.out_stride = out_stride;
  p.n_adapters = lora->n_adapters;
  p.rank = lora->rank;
  p.n = lora->n;
  p.k = lora->k;
  p.m = m;
  p.plan = reinterpret_cast<int32_t*>(static_cast<char*>(workspace_d) + kCounterBytes);
  p.status = status_word(workspace_d);
  p.h = reinterpret_cast<float*>(static_cast<char*>(workspace_d) + kCounterBytes + kLoraPlanBytes);
  p.terms = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace_d) + lora_terms_off(lora, m));
  p.mul = reinterpret_cast<float*>(static_cast<char*>(workspace_d) + lora_mul_off(lora, m));
  p.counters = static_cast<int32_t*>(workspace_d);
  p.splits = lora_splits(lora, m);
  cudaStream_t s = (cudaStream_t)stream;
  const bool bf = lora->dtype == TQ_BF16;
  // tiles: every adapter (and the tokens without one) adds at most one that is not full
  const int per = m > tq::kLoraInBlock ? tq::kLoraTile : tq::kLoraSmall;
  int64_t tiles = (int64_t)(m / per) + lora->n_adapters + 1;
  if (tiles > m) tiles = m;
  if (m > tq::kLoraInBlock)
    return bf ? lora_prompt<true>(p, sms, tiles, s) : lora_prompt<false>(p, sms, tiles, s);
  const dim3 grid((unsigned)tiles * tq::LORA_CLUSTER), block(tq::LORA_THREADS);
  const bool vec = aligned16(y_d) && aligned16(out_d) && y_stride % 4 == 0 && out_stride % 4 == 0;
  if (bf)
    return vec ? launch(tq::lora_kernel<true, true>, grid, block, 0, s, p)
               : launch(tq::lora_kernel<true, false>, grid, block, 0, s, p);
  return vec ? launch(tq::lora_kernel<false, true>, grid, block, 0, s, p)
             : launch(tq::lora_kernel<false, false>, grid, block, 0, s, p);
}

}  // extern "C"
