// C ABI of the operators around a verification (attention over the paged cache, rotary positions with
// the cache write, sampling): argument checks, kernel choice, launches.
#include <cmath>
#include <cstring>
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

// The batch description's checks; `cache`: keys and values are addressed.
spec_status_t check_batch(const spec_paged_batch_t* b, bool cache, int esz) {
  if (!b || b->batch < 0 || b->tokens < 0 || b->kv_heads < 1 || b->dim < 1) return SPEC_ERR_INVALID_ARG;
  if (b->batch > 0 && (!b->cu_q || !b->kv_lens)) return SPEC_ERR_INVALID_ARG;
  if (!cache) return SPEC_OK;
  if (!b->k || !b->v || !b->page_table) return SPEC_ERR_INVALID_ARG;
  if (b->pages < 1 || b->page_size < 1 || b->table_width < 0 || b->table_stride < b->table_width) return SPEC_ERR_INVALID_ARG;
  const long long st[6] = {b->k_page, b->k_token, b->k_head, b->v_page, b->v_token, b->v_head};
  for (long long s : st)
    if (s < 0 || (s * esz) % 16 != 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned(b->k, 16) || !aligned(b->v, 16)) return SPEC_ERR_INVALID_ARG;
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

}  // namespace

extern "C" {

size_t spec_attention_workspace_bytes(int dtype, int q_heads, int kv_heads, int dim, int max_q) {
  return guarded([&]() -> size_t {
    if (!attention_types(dtype) || kv_heads < 1 || q_heads < kv_heads || dim < 8 || dim > 256 || max_q < 0) return 0;
    int sms = 0;
    if (sm_count(&sms) != SPEC_OK) return 0;
    const long long rows = static_cast<long long>(max_q) * (q_heads / kv_heads);
    size_t most = 0;   // over the kernels that rows and dim admit
    for (int kind = 0; kind < 4; ++kind) {
      if ((kind == 0) != (rows <= 16) || (kind >= 2 && (dim < 64 || dim > 128 || (kind == 3) != (rows > 128)))) continue;
      sv::AttnPlan plan;
      if (sv::attention_plan(dtype == SPEC_BF16, kind, 1, dim, sms, &plan) != cudaSuccess) return 0;
      const size_t n = partial_bytes(plan, dim);
      most = n > most ? n : most;
    }
    return kStatusBytes + (most + 255) / 256 * 256;
  }, static_cast<size_t>(0));
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
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_chunk_attention");
    if (!attention_types(dtype) || q_heads < 1 || max_q < 0 || window < 0 || !std::isfinite(scale)) return SPEC_ERR_INVALID_ARG;
    spec_status_t st = check_batch(batch, true, 2);
    if (st != SPEC_OK) return st;
    if (q_heads % batch->kv_heads != 0) return SPEC_ERR_INVALID_ARG;
    if (batch->dim % 8 != 0 || batch->dim > 256) return SPEC_ERR_UNSUPPORTED;
    if (batch->batch == 0 || batch->tokens == 0) return SPEC_OK;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || (q_token * 2) % 16 != 0 || (q_head * 2) % 16 != 0)
      return SPEC_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return SPEC_ERR_WORKSPACE;
    int sms = 0;
    if ((st = sm_count(&sms)) != SPEC_OK) return st;
    const bool bf16 = dtype == SPEC_BF16;
    const int G = q_heads / batch->kv_heads;
    const long long rows = static_cast<long long>(max_q) * G;
    sv::AttnMaps maps;
    int kind = sv::attention_kind(static_cast<int>(rows < 1024 ? rows : 1024), batch->dim, batch->page_size, scale);
    if (kind >= 2 && !sv::attention_maps(bf16, internal_batch(*batch), &maps)) kind = rows <= 16 ? 0 : 1;
    sv::AttnPlan plan;
    if (sv::attention_plan(bf16, kind, static_cast<int>(rows < 1024 ? rows : 1024), batch->dim, sms, &plan) != cudaSuccess)
      return SPEC_ERR_CUDA;
    if (ws_bytes < kStatusBytes + partial_bytes(plan, batch->dim)) return SPEC_ERR_WORKSPACE;
    sv::AttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = internal_batch(*batch);
    p.q = static_cast<const uint8_t*>(q);
    p.q_token = q_token;
    p.q_head = q_head;
    p.out = static_cast<uint8_t*>(out);
    p.lse = out_lse;
    p.Hq = q_heads;
    p.G = G;
    p.G_inv = G > 1 ? ~0ull / G + 1 : 0ull;
    for (p.lanes = 1; p.lanes < 32 && static_cast<long long>(p.lanes) * plan.bm < rows;) p.lanes *= 2;
    p.causal = causal != 0;
    p.window = window;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.status = reinterpret_cast<int32_t*>(ws);
    p.joins = reinterpret_cast<sv::AttnJoin*>(ws + kStatusBytes);
    p.part_ml = reinterpret_cast<float*>(p.joins + plan.grid);
    p.part_o = p.part_ml + static_cast<size_t>(plan.grid) * 2 * plan.bm * 2;
    // an item's fixed cost in key tiles.  Measured, 64 requests x 4 tokens, ragged to 4096 keys (mma.sync):
    // 0: 140, 1: 127, 2: 115, 3: 113, 4: 114 us; 32 x 17 tokens, 64 query heads, ragged to 16384 (tcgen05):
    // 0: 248, 2: 234, 3: 224, 4: 220, 6: 220 us.
    p.overhead = plan.kind >= 2 ? 4 : 3;
    // fewest units worth a CTA: an item's cost and one key tile.  A single token over 1024 keys, 8 key heads
    // (152 units, so 38 CTAs of four): 12.4 us; with two tiles (31 CTAs) 13.3, with four (22) 15.2 us.
    p.min_units = 1 + p.overhead;
    const long long wait_us = tuning ? tuning->wait_limit_us : 0;
    p.wait_limit = wait_us == 0 ? kWaitNs : wait_us < 0 ? 0 : wait_us < kWaitNs ? wait_us * 1000 : kWaitNs * 1000;
    p.n_max = plan.grid;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The two kernels talk through the workspace: another thread's call with the same one must not come between.
    static std::mutex pair;
    std::lock_guard<std::mutex> lk(pair);
    if (sv::launch_attention(bf16, plan, p, maps, s) != cudaSuccess) return SPEC_ERR_CUDA;
    return sv::launch_attention_combine(bf16, plan, p, s) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  }, SPEC_ERR_CUDA);
}

spec_status_t spec_rope_append(const spec_rope_tensors_t* t, int dtype, int q_heads, const spec_paged_batch_t* batch,
                               const unsigned long long* freq, int rotary_dim, float factor, int interleaved,
                               void* workspace, void* stream) {
  return guarded([&]() -> spec_status_t {
    const sv::ApiRange range("spec_rope_append");
    if (!t || (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) || q_heads < 0) return SPEC_ERR_INVALID_ARG;
    const bool cache = batch && batch->k;
    spec_status_t st = check_batch(batch, cache, dtype == SPEC_F32 ? 4 : 2);
    if (st != SPEC_OK) return st;
    if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > batch->dim || !std::isfinite(factor)) return SPEC_ERR_INVALID_ARG;
    if (batch->dim > 1024) return SPEC_ERR_UNSUPPORTED;
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
    return sv::launch_rope(dtype, p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
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
