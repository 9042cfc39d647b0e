// Declarations shared by the kernels and the host code of the operators around a verification:
// paged-cache attention, rotary positions with the cache write, and sampling.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace sv {

// Status bit (with those of spec_internal.h): a page id outside the cache, or a position beyond the page table.
constexpr int kStatusPageRange = 4;

// A batch of requests over a paged cache.  Strides are in elements.
struct PagedBatch {
  uint8_t* k;
  uint8_t* v;
  long long k_page, k_token, k_head, v_page, v_token, v_head;
  const int32_t* table;      // [B, table_width], rows table_stride apart
  long long table_stride;
  int table_width, pages, page_size;
  const int32_t* kv_lens;    // [B] cached tokens, the new ones included
  const int32_t* cu_q;       // [B + 1] first new token of every request
  int B, N;                  // requests, new tokens
  int Hkv, D;
};

// The item that begins in a CTA's run and goes on in others': what the combine kernel joins.
struct alignas(16) AttnJoin {
  int rows, row0;            // rows of the item (0: no such item), first row
  int token0, head0;         // the request's first new token, the key head's first query head
  int last;                  // last CTA that works on it
  int slot;                  // this CTA's partial
  int pad[2];
};

struct AttnParams {
  PagedBatch c;
  const uint8_t* q;
  long long q_token, q_head;
  uint8_t* out;              // [N, Hq, D]
  float* lse;                // [N, Hq] or null
  int Hq, G;                 // query heads, query heads per key head
  unsigned long long G_inv;  // ceil(2^64 / G), 0 for G = 1
  int lanes;                 // threads that share a request's row tiles when the work is divided
  int causal, window;
  float scale_log2;          // softmax scale x log2(e)
  float* part_o;             // [2 n, BM, D] partial rows of items that more than one CTA works on
  float* part_ml;            // [2 n, BM, 2] their maximum and sum
  AttnJoin* joins;           // [n]
  int overhead;              // an item's cost beside its key tiles, in key tiles
  int min_units;             // fewest units worth a CTA of their own
  int n_max;                 // CTAs launched
  long long wait_limit;      // ns per bounded wait (tcgen05 kernel); 0: the first one gives up at once
  int32_t* status;
};

// Kernel families of the attention: rows per tile, keys per tile.
struct AttnPlan {
  int kind;                  // 0: 16-row tiles, 1: 64-row tiles (mma.sync); 2, 3: 128- and 256-row tiles (tcgen05)
  int bm, bn, grid, smem, dp;
  int rows;                  // the most rows of an item that the caller's bound allows
};

// TMA descriptors of the two caches.
struct AttnMaps {
  alignas(64) uint8_t k[128];
  alignas(64) uint8_t v[128];
};

int attention_kind(int rows, int D, int page_size, float scale);
cudaError_t attention_plan(bool bf16, int kind, int rows, int D, int sms, AttnPlan* plan);
bool attention_maps(bool bf16, const PagedBatch& c, AttnMaps* maps);   // false: TMA cannot describe the caches
cudaError_t launch_attention(bool bf16, const AttnPlan& plan, const AttnParams& p, const AttnMaps& maps, cudaStream_t stream);
cudaError_t launch_attention_combine(bool bf16, const AttnPlan& plan, const AttnParams& p, cudaStream_t stream);

struct RopeParams {
  PagedBatch c;              // k / v may be null: nothing is stored
  const uint8_t *q, *k, *v;  // new tokens
  uint8_t *q_out, *k_out;    // rotated queries; rotated keys (or null)
  long long q_token, q_head, k_token, k_head, v_token, v_head, qo_token, qo_head, ko_token, ko_head;
  const unsigned long long* freq;  // [rotary / 2] turns a position x 2^64
  float factor;
  int Hq, rotary, interleaved;
  int32_t* status;
};
cudaError_t launch_rope(int dtype, const RopeParams& p, int sms, cudaStream_t stream);

struct SampleParams {
  const void* logits;
  long long stride;
  int R, V;
  const float* uniforms;
  const float *temperature, *top_p, *min_p;   // per row, or null: the scalars
  const int32_t* top_k;
  float temperature0, top_p0, min_p0;
  int top_k0;
  int32_t* tokens;
  float* probs;
  int32_t* kept;
  void* filtered;
  long long filtered_stride;
};
cudaError_t launch_sample(int dtype, const SampleParams& p, int sms, cudaStream_t stream);

}  // namespace sv
