// C ABI of the operators around a verification (attention over the paged cache, rotary positions with
// the cache write, sampling): argument checks, kernel choice, launches.
#include <cmath>
#include <cstring>
#include <initializer_list>
#include <map>
#include <mutex>

#include "../../include/spec_verify.h"
#include "api_range.h"
#include "spec_internal.h"
#include "step_internal.h"

namespace {

constexpr size_t kStatusBytes = 256;
constexpr int kMaxSampleV = 262144;
constexpr long long kWaitNs = 2000000000ll;   // wall time per bounded on-device wait

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// SM count of the current device (cached).
spec_status_t sm_count(int* sms) {
  static std::mutex mu;
  static std::map<int, int> cache;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  auto it = cache.find(dev);
  if (it == cache.end()) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SPEC_ERR_CUDA;
    it = cache.emplace(dev, n).first;
  }
  *sms = it->second;
  return SPEC_OK;
}

size_t partial_bytes(const sv::AttnPlan& plan, int D) {
  return static_cast<size_t>(plan.grid) * (sizeof(sv::AttnJoin) + 2 * plan.bm * (D + 2) * sizeof(float));
}

// The batch description's checks; `cache`: keys and values are addressed, whose bases and strides (in units of
// `esz` bytes) are multiples of `align` bytes.
spec_status_t check_batch(const spec_paged_batch_t* b, bool cache, int esz, int align = 16) {
  if (!b || b->batch < 0 || b->tokens < 0 || b->kv_heads < 1 || b->dim < 1) return SPEC_ERR_INVALID_ARG;
  if (b->batch > 0 && (!b->cu_q || !b->kv_lens)) return SPEC_ERR_INVALID_ARG;
  if (!cache) return SPEC_OK;
  if (!b->k || !b->v || !b->page_table) return SPEC_ERR_INVALID_ARG;
  if (b->pages < 1 || b->page_size < 1 || b->table_width < 0 || b->table_stride < b->table_width) return SPEC_ERR_INVALID_ARG;
  const long long st[6] = {b->k_page, b->k_token, b->k_head, b->v_page, b->v_token, b->v_head};
  for (long long s : st)
    if (s < 0 || (s * esz) % align != 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned(b->k, align) || !aligned(b->v, align)) return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

sv::PagedBatch internal_batch(const spec_paged_batch_t& b) {
  sv::PagedBatch c;
  c.k = static_cast<uint8_t*>(b.k);
  c.v = static_cast<uint8_t*>(b.v);
  c.k_page = b.k_page;
  c.k_token = b.k_token;
  c.k_head = b.k_head;
  c.v_page = b.v_page;
  c.v_token = b.v_token;
  c.v_head = b.v_head;
  c.table = b.page_table;
  c.table_stride = b.table_stride;
  c.table_width = b.table_width;
  c.pages = b.pages;
  c.page_size = b.page_size;
  c.kv_lens = b.kv_lens;
  c.cu_q = b.cu_q;
  c.B = b.batch;
  c.N = b.tokens;
  c.Hkv = b.kv_heads;
  c.D = b.dim;
  return c;
}

// A power of two between 2^-64 and 2^64.
bool fp4_unit(float u) {
  int e = 0;
  return std::isfinite(u) && std::frexp(u, &e) == 0.5f && e >= -63 && e <= 65;
}

spec_status_t check_scales(const spec_paged_batch_t* b, const spec_fp4_scales_t* s) {
  if (!s || !s->k || !s->v || !fp4_unit(s->k_unit) || !fp4_unit(s->v_unit)) return SPEC_ERR_INVALID_ARG;
  for (long long x : {s->k_page, s->k_token, s->k_head, s->v_page, s->v_token, s->v_head})
    if (x < 0) return SPEC_ERR_INVALID_ARG;
  return b->dim % 16 != 0 || b->dim > 256 ? SPEC_ERR_UNSUPPORTED : SPEC_OK;
}

sv::Fp4Scales internal_scales(const spec_paged_batch_t& b, const spec_fp4_scales_t& f) {
  sv::Fp4Scales s;
  s.k = static_cast<uint8_t*>(f.k);
  s.v = static_cast<uint8_t*>(f.v);
  s.k_page = f.k_page;
  s.k_token = f.k_token;
  s.k_head = f.k_head;
  s.v_page = f.v_page;
  s.v_token = f.v_token;
  s.v_head = f.v_head;
  bool whole = (b.dim == 64 || b.dim == 128 || b.dim == 256) && aligned(b.k, 16) && aligned(b.v, 16) &&
               aligned(f.k, b.dim / 16) && aligned(f.v, b.dim / 16);
  for (long long x : {b.k_page, b.k_token, b.k_head, b.v_page, b.v_token, b.v_head}) whole = whole && x % 16 == 0;
  for (long long x : {f.k_page, f.k_token, f.k_head, f.v_page, f.v_token, f.v_head}) whole = whole && x % (b.dim / 16) == 0;
  s.whole = whole;
  // whatever page, slot and head: within (pages - 1) page + (page_size - 1) token + (heads - 1) head bytes of the base
  const long long most = 1ll << 32;
  s.alike = f.k_page < most && f.k_token < most && f.k_head < most && f.k_page == f.v_page && f.k_token == f.v_token &&
            f.k_head == f.v_head && b.k_page == 8 * f.k_page && b.k_token == 8 * f.k_token && b.k_head == 8 * f.k_head &&
            b.v_page == b.k_page && b.v_token == b.k_token && b.v_head == b.k_head &&
            static_cast<double>(b.pages - 1) * f.k_page + static_cast<double>(b.page_size - 1) * f.k_token +
                    static_cast<double>(b.kv_heads - 1) * f.k_head < static_cast<double>(most - 1);
  return s;
}

bool attention_types(int dtype) { return dtype == SPEC_BF16 || dtype == SPEC_F16; }

// No C++ exception (a lock or a cache entry that cannot be had) leaves a C entry.
template <typename F>
auto guarded(F f, decltype(f()) failed) -> decltype(f()) {
  try {
    return f();
  } catch (...) {
    return failed;
  }
}

size_t attention_workspace(int dtype, int q_heads, int kv_heads, int dim, int max_q, bool fp4) {
  if (!attention_types(dtype) || kv_heads < 1 || q_heads < kv_heads || dim < 8 || dim > 256 || max_q < 0) return 0;
  if (fp4 && dim % 16 != 0) return 0;
  int sms = 0;
  if (sm_count(&sms) != SPEC_OK) return 0;
  const long long rows = static_cast<long long>(max_q) * (q_heads / kv_heads);
  size_t most = 0;   // over the kernels that rows and dim admit
  for (int kind = 0; kind < 4; ++kind) {
    if (!fp4 && ((kind == 0) != (rows <= 16) || (kind >= 2 && (dim < 64 || dim > 128 || (kind == 3) != (rows > 128))))) continue;
    if (fp4 && kind != sv::attention_fp4_kind(static_cast<int>(rows < 1024 ? rows : 1024), dim, 1.f) && kind != 0) continue;
    for (int variant = 0; variant < (fp4 ? 3 : 2); ++variant) {   // first tokens kept or not; over 4 bits, tiles of 8, 16, 32 rows
      sv::AttnPlan plan;
      if (sv::attention_plan({dtype == SPEC_BF16, !fp4 && variant, fp4, true}, kind, fp4 ? 8 << variant : 1, dim, sms, &plan) !=
          cudaSuccess)
        return 0;
      const size_t n = partial_bytes(plan, dim);
      most = n > most ? n : most;
    }
  }
  return kStatusBytes + (most + 255) / 256 * 256;
}

struct AttentionCall {
  const void* q;
  long long q_token, q_head;
  int dtype, q_heads;
  const spec_paged_batch_t* batch;
  const spec_fp4_scales_t* scales;   // null: the cache has q's type
  int max_q;
  float scale;
  int causal, window, sinks;
  void* out;
  float* lse;
  void* workspace;
  size_t ws_bytes;
  cudaStream_t stream;
  const spec_tuning_t* tuning;
};

// Kernels that talk through a workspace: another thread's call with the same one must not come between a call's launches.
std::mutex g_pair;

spec_status_t run_attention(const AttentionCall& a) {
  const spec_paged_batch_t* batch = a.batch;
  const bool fp4 = a.scales != nullptr;
  if (!attention_types(a.dtype) || a.q_heads < 1 || a.max_q < 0 || a.window < 0 || a.sinks < 0 || !std::isfinite(a.scale))
    return SPEC_ERR_INVALID_ARG;
  spec_status_t st = fp4 ? check_batch(batch, true, 1, 8) : check_batch(batch, true, 2);
  if (st != SPEC_OK) return st;
  if (a.q_heads % batch->kv_heads != 0) return SPEC_ERR_INVALID_ARG;
  if (batch->dim % 8 != 0 || batch->dim > 256) return SPEC_ERR_UNSUPPORTED;
  if (fp4 && (st = check_scales(batch, a.scales)) != SPEC_OK) return st;
  if (batch->batch == 0 || batch->tokens == 0) return SPEC_OK;
  if (!a.q || !a.out || !aligned(a.q, 16) || !aligned(a.out, 16) || (a.q_token * 2) % 16 != 0 || (a.q_head * 2) % 16 != 0)
    return SPEC_ERR_INVALID_ARG;
  if (!a.workspace || !aligned(a.workspace, 256)) return SPEC_ERR_WORKSPACE;
  int sms = 0;
  if ((st = sm_count(&sms)) != SPEC_OK) return st;
  const int G = a.q_heads / batch->kv_heads;
  const long long all_rows = static_cast<long long>(a.max_q) * G;
  const int rows = static_cast<int>(all_rows < 1024 ? all_rows : 1024);
  sv::AttnMaps maps = {};
  sv::Fp4Scales scales = {};
  if (fp4) scales = internal_scales(*batch, *a.scales);
  const sv::AttnForm form = {a.dtype == SPEC_BF16, a.window > 0 && a.sinks > 0, fp4, scales.whole != 0};
  // strides that are not alike (keys' and values', or codes' and scales') leave the kernel that reads a key's 8 bytes and its
  // scales one by one: 32 x 17 tokens ragged to 16384 keys 1297 us for 242, 64 single tokens to 8192 keys 199 for 73.  (Heads other
  // than 64, 128 and 256 long take the same reads there whatever their strides: 64 single tokens of heads of 80 134-138.)
  int kind = fp4 ? (scales.alike ? sv::attention_fp4_kind(rows, batch->dim, a.scale) : 0) : sv::attention_kind(rows, batch->dim, batch->page_size, a.scale);
  if (!fp4 && kind >= 2 && !sv::attention_maps(form.bf16, internal_batch(*batch), &maps)) kind = rows <= 16 ? 0 : 1;
  sv::AttnPlan plan;
  if (sv::attention_plan(form, kind, rows, batch->dim, sms, &plan) != cudaSuccess) return SPEC_ERR_CUDA;
  if (a.ws_bytes < kStatusBytes + partial_bytes(plan, batch->dim)) return SPEC_ERR_WORKSPACE;
  sv::AttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = internal_batch(*batch);
  p.q = static_cast<const uint8_t*>(a.q);
  p.q_token = a.q_token;
  p.q_head = a.q_head;
  p.out = static_cast<uint8_t*>(a.out);
  p.lse = a.lse;
  p.Hq = a.q_heads;
  p.G = G;
  p.G_inv = G > 1 ? ~0ull / G + 1 : 0ull;
  for (p.lanes = 1; p.lanes < 32 && static_cast<long long>(p.lanes) * plan.bm < all_rows;) p.lanes *= 2;
  p.causal = a.causal != 0;
  p.window = a.window;
  p.sinks = form.sinks ? a.sinks : 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634 * (fp4 ? a.scales->k_unit : 1.f));
  if (!std::isfinite(p.scale_log2)) return SPEC_ERR_INVALID_ARG;
  p.v_unit = fp4 ? a.scales->v_unit : 1.f;
  p.s = scales;
  p.page_inv = batch->page_size > 1 ? static_cast<unsigned>((1ull << 32) / batch->page_size) : 0xffffffffu;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  p.status = reinterpret_cast<int32_t*>(ws);
  p.joins = reinterpret_cast<sv::AttnJoin*>(ws + kStatusBytes);
  p.part_ml = reinterpret_cast<float*>(p.joins + plan.grid);
  p.part_o = p.part_ml + static_cast<size_t>(plan.grid) * 2 * plan.bm * 2;
  // an item's fixed cost in key tiles.  Measured, 64 requests x 4 tokens, ragged to 4096 keys (mma.sync):
  // 0: 140, 1: 127, 2: 115, 3: 113, 4: 114 us; 32 x 17 tokens, 64 query heads, ragged to 16384 (tcgen05):
  // 0: 248, 2: 234, 3: 224, 4: 220, 6: 220 us.  Over 4 bits (the same 32 x 17 tokens, tcgen05): 1: 294, 2: 282, 3: 257, 4: 245,
  // 5: 242 us; 64 single tokens to 16384 keys (mma.sync): 1: 139, 2: 134, 3: 130, 4: 131, 6: 132 us.
  p.overhead = plan.kind >= 2 ? (fp4 ? 5 : 4) : 3;
  // fewest units worth a CTA: an item's cost and one key tile.  A single token over 1024 keys, 8 key heads
  // (152 units, so 38 CTAs of four): 12.4 us; with two tiles (31 CTAs) 13.3, with four (22) 15.2 us.
  p.min_units = 1 + p.overhead;
  const long long wait_us = a.tuning ? a.tuning->wait_limit_us : 0;
  p.wait_limit = wait_us == 0 ? kWaitNs : wait_us < 0 ? 0 : wait_us < kWaitNs ? wait_us * 1000 : kWaitNs * 1000;
  p.n_max = plan.grid;
  std::lock_guard<std::mutex> lk(g_pair);
  if (sv::launch_attention(form, plan, p, maps, a.stream) != cudaSuccess) return SPEC_ERR_CUDA;
  return sv::launch_attention_combine(form.bf16, plan, p, a.stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// rope_append's call, into a cache of the tokens' type or (scales) one held in 4 bits.
spec_status_t run_rope(const spec_rope_tensors_t* t, int dtype, int q_heads, const spec_paged_batch_t* batch,
                       const spec_fp4_scales_t* scales, const unsigned long long* freq, int rotary_dim, float factor,
                       int interleaved, void* workspace, cudaStream_t stream) {
  const bool fp4 = scales != nullptr;
  if (!t || (dtype != SPEC_BF16 && dtype != SPEC_F16 && (fp4 || dtype != SPEC_F32)) || q_heads < 0) return SPEC_ERR_INVALID_ARG;
  const bool cache = fp4 || (batch && batch->k);
  spec_status_t st = fp4 ? check_batch(batch, true, 1, 8) : check_batch(batch, cache, dtype == SPEC_F32 ? 4 : 2);
  if (st != SPEC_OK) return st;
  if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > batch->dim || !std::isfinite(factor)) return SPEC_ERR_INVALID_ARG;
  if (batch->dim > 1024) return SPEC_ERR_UNSUPPORTED;
  if (fp4 && (st = check_scales(batch, scales)) != SPEC_OK) return st;
  if (batch->batch == 0 || batch->tokens == 0) return SPEC_OK;
  if ((q_heads > 0 && (!t->q || !t->q_out)) || !t->k || (cache && !t->v) || (rotary_dim > 0 && !freq))
    return SPEC_ERR_INVALID_ARG;
  if (!cache && !t->k_out) return SPEC_ERR_INVALID_ARG;
  if (cache && (!workspace || !aligned(workspace, 256))) return SPEC_ERR_WORKSPACE;
  sv::RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = internal_batch(*batch);
  p.q = static_cast<const uint8_t*>(t->q);
  p.k = static_cast<const uint8_t*>(t->k);
  p.v = static_cast<const uint8_t*>(t->v);
  p.q_out = static_cast<uint8_t*>(t->q_out);
  p.k_out = static_cast<uint8_t*>(t->k_out);
  p.q_token = t->q_token;
  p.q_head = t->q_head;
  p.k_token = t->k_token;
  p.k_head = t->k_head;
  p.v_token = t->v_token;
  p.v_head = t->v_head;
  p.qo_token = t->q_out_token;
  p.qo_head = t->q_out_head;
  p.ko_token = t->k_out_token;
  p.ko_head = t->k_out_head;
  p.freq = freq;
  p.factor = factor;
  p.Hq = q_heads;
  p.rotary = rotary_dim;
  p.interleaved = interleaved != 0;
  p.status = static_cast<int32_t*>(workspace);
  int sms = 0;
  if ((st = sm_count(&sms)) != SPEC_OK) return st;
  if (fp4)
    return sv::launch_rope_fp4(dtype, p, internal_scales(*batch, *scales), scales->k_unit, scales->v_unit, sms, stream) == cudaSuccess
               ? SPEC_OK : SPEC_ERR_CUDA;
  return sv::launch_rope(dtype, p, sms, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// Entries of a table, and pages: the page kernels count both in 32 bits, in steps of up to 1024 beyond the last one.
constexpr long long kMaxPageEntries = 1ll << 30;

// Workspace of the page operators: ints behind the status.
size_t pages_ints(int pages, int rows) {
  const size_t copies = static_cast<size_t>(rows > pages / 2 ? rows : pages / 2);
  return 16 + 4 * static_cast<size_t>(rows) + 2 * copies + 2 * static_cast<size_t>(pages);
}

spec_status_t run_pages(bool compact, const spec_page_pool_t* pool, int page_size, const int32_t* table, long long stride,
                        int rows, int width, const int32_t* lens, const int32_t* kept, const int32_t* parents,
                        int32_t* out_table, long long out_stride, int32_t* out_used, void* workspace, size_t ws_bytes,
                        cudaStream_t stream) {
  if (!pool || pool->pages < 1 || pool->n_arrays < 0 || pool->max_bytes < 0 || (pool->n_arrays > 0 && !pool->arrays))
    return SPEC_ERR_INVALID_ARG;
  if (rows < 0 || width < 0 || stride < width || out_stride < width || page_size < 1) return SPEC_ERR_INVALID_ARG;
  if (static_cast<long long>(rows) * width > kMaxPageEntries || rows > kMaxPageEntries || pool->pages > kMaxPageEntries ||
      pool->max_bytes > (1ll << 40))
    return SPEC_ERR_UNSUPPORTED;
  const bool empty = rows == 0 || width == 0;
  if (empty && !compact) return SPEC_OK;
  if ((!empty && (!table || !out_table)) || (compact ? !out_used : !lens || !kept)) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < kStatusBytes + 4 * pages_ints(pool->pages, rows))
    return SPEC_ERR_WORKSPACE;
  sv::PageParams p;
  std::memset(&p, 0, sizeof(p));
  p.arrays = reinterpret_cast<const sv::PageArray*>(pool->arrays);
  p.n_arrays = pool->n_arrays;
  p.pages = pool->pages;
  p.page_size = page_size;
  p.table = table;
  p.stride = stride;
  p.rows = rows;
  p.width = width;
  p.lens = lens;
  p.kept = kept;
  p.parents = parents;
  p.out = out_table;
  p.out_stride = out_stride;
  p.used = out_used;
  p.status = static_cast<int32_t*>(workspace);
  int* ws = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
  const int copies = rows > p.pages / 2 ? rows : p.pages / 2;
  p.counts = ws;
  p.moves = ws + 8;
  p.wanted = ws + 9;
  p.plan = reinterpret_cast<int4*>(ws + 16);
  p.src = ws + 16 + 4 * static_cast<size_t>(rows);
  p.dst = p.src + copies;
  p.list = p.dst + copies;
  p.mark = p.list + p.pages;
  int sms = 0;
  const spec_status_t st = sm_count(&sms);
  if (st != SPEC_OK) return st;
  std::lock_guard<std::mutex> lk(g_pair);
  return sv::launch_pages(compact, p, pool->max_bytes, sms, stream) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t spec_attention_workspace_bytes(int dtype, int q_heads, int kv_heads, int dim, int max_q) {
  return guarded([&] { return attention_workspace(dtype, q_heads, kv_heads, dim, max_q, false); }, static_cast<size_t>(0));
}

size_t spec_attention_fp4_workspace_bytes(int dtype, int q_heads, int kv_heads, int dim, int max_q) {
  return guarded([&] { return attention_workspace(dtype, q_heads, kv_heads, dim, max_q, true); }, static_cast<size_t>(0));
}

spec_status_t spec_chunk_attention(const void* q, long long q_token, long long q_head, int dtype, int q_heads,
                                   const spec_paged_batch_t* batch, int max_q, float scale, int causal, int window,
                                   void* out, float* out_lse, void* workspace, size_t ws_bytes, void* stream) {
  return spec_chunk_attention_tuned(q, q_token, q_head, dtype, q_heads, batch, max_q, scale, causal, window, out, out_lse,
                                    workspace, ws_bytes, stream, nullptr);
}

spec_status_t spec_chunk_attention_tuned(const void* q, long long q_token, long long q_head, int dtype, int q_heads,
                                         const spec_paged_batch_t* batch, int max_q, float scale, int causal, int window,
                                         void* out, float* out_lse, void* workspace, size_t ws_bytes, void* stream,
                                         const spec_tuning_t* tuning) {
  return spec_chunk_attention_sinks(q, q_token, q_head, dtype, q_heads, batch, max_q, scale, causal, window, 0, out, out_lse,
                                    workspace, ws_bytes, stream, tuning);
}

spec_status_t spec_chunk_attention_sinks(const void* q, long long q_token, long long q_head, int dtype, int q_heads,
                                         const spec_paged_batch_t* batch, int max_q, float scale, int causal, int window,
                                         int sinks, void* out, float* out_lse, void* workspace, size_t ws_bytes,
                                         void* stream, const spec_tuning_t* tuning) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_chunk_attention");
    return run_attention({q, q_token, q_head, dtype, q_heads, batch, nullptr, max_q, scale, causal, window, sinks, out, out_lse,
                          workspace, ws_bytes, static_cast<cudaStream_t>(stream), tuning});
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_chunk_attention_fp4(const void* q, long long q_token, long long q_head, int dtype, int q_heads,
                                       const spec_paged_batch_t* batch, const spec_fp4_scales_t* scales, int max_q,
                                       float scale, int causal, int window, int sinks, void* out, float* out_lse,
                                       void* workspace, size_t ws_bytes, void* stream, const spec_tuning_t* tuning) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_chunk_attention_fp4");
    if (!scales) return SPEC_ERR_INVALID_ARG;
    return run_attention({q, q_token, q_head, dtype, q_heads, batch, scales, max_q, scale, causal, window, sinks, out, out_lse,
                          workspace, ws_bytes, static_cast<cudaStream_t>(stream), tuning});
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_rope_append(const spec_rope_tensors_t* t, int dtype, int q_heads, const spec_paged_batch_t* batch,
                               const unsigned long long* freq, int rotary_dim, float factor, int interleaved,
                               void* workspace, void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_rope_append");
    return run_rope(t, dtype, q_heads, batch, nullptr, freq, rotary_dim, factor, interleaved, workspace,
                    static_cast<cudaStream_t>(stream));
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_rope_append_fp4(const spec_rope_tensors_t* t, int dtype, int q_heads, const spec_paged_batch_t* batch,
                                   const spec_fp4_scales_t* scales, const unsigned long long* freq, int rotary_dim,
                                   float factor, int interleaved, void* workspace, void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_rope_append_fp4");
    if (!scales) return SPEC_ERR_INVALID_ARG;
    return run_rope(t, dtype, q_heads, batch, scales, freq, rotary_dim, factor, interleaved, workspace,
                    static_cast<cudaStream_t>(stream));
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_fp4_values(const void* codes, long long page, long long token, long long head, const void* scales,
                              long long s_page, long long s_token, long long s_head, float unit, int pages,
                              int page_size, int heads, int dim, int dtype, void* out, void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_fp4_values");
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (pages < 0 || page_size < 1 || heads < 1 || dim < 1 || !fp4_unit(unit)) return SPEC_ERR_INVALID_ARG;
    if (dim % 16 != 0 || dim > 256) return SPEC_ERR_UNSUPPORTED;
    for (long long x : {page, token, head})
      if (x < 0 || x % 8 != 0) return SPEC_ERR_INVALID_ARG;
    for (long long x : {s_page, s_token, s_head})
      if (x < 0) return SPEC_ERR_INVALID_ARG;
    if (pages == 0) return SPEC_OK;
    if (!codes || !scales || !out || !aligned(codes, 8) || !aligned(out, 16)) return SPEC_ERR_INVALID_ARG;
    int sms = 0;
    const spec_status_t st = sm_count(&sms);
    if (st != SPEC_OK) return st;
    const sv::Fp4Values p = {static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), page, token, head,
                             s_page, s_token, s_head, unit, pages, page_size, heads, dim, out};
    return sv::launch_fp4_values(dtype, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  }, SPEC_ERR_CUDA);
}

size_t spec_pages_workspace_bytes(int pages, int rows) {
  if (pages < 1 || rows < 0 || pages > kMaxPageEntries || rows > kMaxPageEntries) return 0;
  return kStatusBytes + (4 * pages_ints(pages, rows) + 255) / 256 * 256;
}

spec_status_t spec_assign_pages(const spec_page_pool_t* pool, int page_size, const int32_t* table, long long table_stride,
                                int rows, int width, const int32_t* lens, const int32_t* kept, const int32_t* parents,
                                int32_t* out_table, long long out_stride, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_assign_pages");
    return run_pages(false, pool, page_size, table, table_stride, rows, width, lens, kept, parents, out_table, out_stride,
                     nullptr, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_compact_pages(const spec_page_pool_t* pool, const int32_t* table, long long table_stride, int rows,
                                 int width, int32_t* out_table, long long out_stride, int32_t* out_used, void* workspace,
                                 size_t ws_bytes, void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_compact_pages");
    return run_pages(true, pool, 1, table, table_stride, rows, width, nullptr, nullptr, nullptr, out_table, out_stride,
                     out_used, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_sample_tokens(const void* logits, long long row_stride, int dtype, int rows, int V,
                                 const float* uniforms, const spec_sampling_t* how, int32_t* out_tokens,
                                 float* out_probs, int32_t* out_kept, void* out_filtered, long long filtered_stride,
                                 void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_sample_tokens");
    if ((dtype != SPEC_F32 && dtype != SPEC_BF16) || rows < 0 || V < 1 || !how) return SPEC_ERR_INVALID_ARG;
    if (V > kMaxSampleV) return SPEC_ERR_UNSUPPORTED;
    if (!how->temperature_rows && (!(how->temperature >= 0.f))) return SPEC_ERR_INVALID_ARG;
    if (!how->top_p_rows && std::isnan(how->top_p)) return SPEC_ERR_INVALID_ARG;
    if (!how->min_p_rows && std::isnan(how->min_p)) return SPEC_ERR_INVALID_ARG;
    if (row_stride < V || (out_filtered && filtered_stride < V)) return SPEC_ERR_INVALID_ARG;
    if (rows == 0) return SPEC_OK;
    if (!logits || !uniforms || !out_tokens) return SPEC_ERR_INVALID_ARG;
    sv::SampleParams p;
    p.logits = logits;
    p.stride = row_stride;
    p.R = rows;
    p.V = V;
    p.uniforms = uniforms;
    p.temperature = how->temperature_rows;
    p.top_p = how->top_p_rows;
    p.min_p = how->min_p_rows;
    p.top_k = how->top_k_rows;
    p.temperature0 = how->temperature;
    p.top_p0 = how->top_p;
    p.min_p0 = how->min_p;
    p.top_k0 = how->top_k;
    p.tokens = out_tokens;
    p.probs = out_probs;
    p.kept = out_kept;
    p.filtered = out_filtered;
    p.filtered_stride = filtered_stride;
    int sms = 0;
    const spec_status_t st = sm_count(&sms);
    if (st != SPEC_OK) return st;
    return sv::launch_sample(dtype, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  }, SPEC_ERR_CUDA);
}

}  // extern "C"
