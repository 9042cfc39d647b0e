// Host side of the paged attention (kernel choice, launches) and the kernel that joins items split
// over several CTAs.
#include <map>
#include <mutex>
#include <tuple>

#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_mma_fn<true, false>(int dp, int bm);
template <>
const void* attn_mma_fn<false, false>(int dp, int bm);
template <>
const void* attn_mma_fn<true, true>(int dp, int bm);
template <>
const void* attn_mma_fn<false, true>(int dp, int bm);
template <>
const void* attn_tc_fn<true, false>(int dp, bool wide);
template <>
const void* attn_tc_fn<false, false>(int dp, bool wide);
template <>
const void* attn_tc_fn<true, true>(int dp, bool wide);
template <>
const void* attn_tc_fn<false, true>(int dp, bool wide);
template <>
const void* attn_tc_fp4_fn<true>(int dp, bool wide, bool whole);
template <>
const void* attn_tc_fp4_fn<false>(int dp, bool wide, bool whole);
template <>
const void* attn_fp4_fn<true>(int dp, int bm);
template <>
const void* attn_fp4_fn<false>(int dp, int bm);

// Joins the item that CTA blockIdx.x left a record of: one warp per row, the partials in key order,
// each scaled by 2^(its maximum - the largest).  fp32.
template <bool BF16>
__global__ void __launch_bounds__(128) attn_combine_kernel(const AttnParams p, int bm) {
  using A = AttnType<BF16>;
  const int c1 = blockIdx.x, lane = threadIdx.x & 31, D = p.c.D;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const AttnJoin j = p.joins[c1];
  for (int r = blockIdx.y * 4 + threadIdx.x / 32; r < j.rows; r += gridDim.y * 4) {
    auto slot = [&](int c) { return static_cast<long long>(c == c1 ? j.slot : 2 * c) * bm + r; };
    float m = ninf();
    for (int c = c1 + lane; c <= j.last; c += 32) m = fmaxf(m, __ldcg(p.part_ml + slot(c) * 2));
    m = warp_maxf(m);
    const float ref = m == ninf() ? 0.f : m;
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    float l = 0.f;
#pragma unroll 8
    for (int c = c1; c <= j.last; ++c) {
      const long long s = slot(c);
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + s * 2));
      const float f = ex2(ml.x - ref);
      l += f * ml.y;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = lane * 4 + i * 128;
        if (d < D) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(p.part_o + s * D + d));
          acc[i].x += f * x.x;
          acc[i].y += f * x.y;
          acc[i].z += f * x.z;
          acc[i].w += f * x.w;
        }
      }
    }
    const float inv = attn_factor(l, p.v_unit);
    const int tok = attn_token(p, j.row0 + r);
    const long long row = static_cast<long long>(j.token0 + tok) * p.Hq + j.head0 + (j.row0 + r - tok * p.G);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = lane * 4 + i * 128;
      if (d < D)
        *reinterpret_cast<uint2*>(p.out + (row * D + d) * 2) =
            make_uint2(A::pack(acc[i].x * inv, acc[i].y * inv), A::pack(acc[i].z * inv, acc[i].w * inv));
    }
    if (lane == 0 && p.lse) p.lse[row] = attn_lse(m, l);
  }
}

namespace {
std::mutex g_mu;
std::map<std::tuple<int, const void*>, int> g_occ;   // resident CTAs per SM, attributes set
}  // namespace

// Resident CTAs per SM of a kernel with this much dynamic shared memory (attributes set once per device).
static cudaError_t resident(const void* fn, int threads, int smem, int* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_occ.find({dev, fn});
  if (it == g_occ.end()) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem);
    if (e != cudaSuccess) return e;
    it = g_occ.emplace(std::make_tuple(dev, fn), n > 0 ? n : 1).first;
  }
  *out = it->second;
  return cudaSuccess;
}

template <bool BF16, bool SINKS>
static const void* kernel_of(const AttnPlan& plan) {
  return plan.kind >= 2 ? attn_tc_fn<BF16, SINKS>(plan.dp, plan.kind == 3) : attn_mma_fn<BF16, SINKS>(plan.dp, plan.bm);
}
static const void* kernel_of(const AttnForm& form, const AttnPlan& plan) {
  if (form.fp4 && plan.kind >= 2)
    return form.bf16 ? attn_tc_fp4_fn<true>(plan.dp, plan.kind == 3, form.whole) : attn_tc_fp4_fn<false>(plan.dp, plan.kind == 3, form.whole);
  if (form.fp4) return form.bf16 ? attn_fp4_fn<true>(plan.dp, plan.bm) : attn_fp4_fn<false>(plan.dp, plan.bm);
  if (form.sinks) return form.bf16 ? kernel_of<true, true>(plan) : kernel_of<false, true>(plan);
  return form.bf16 ? kernel_of<true, false>(plan) : kernel_of<false, false>(plan);
}

cudaError_t attention_plan(const AttnForm& form, int kind, int rows, int D, int sms, AttnPlan* plan) {
  plan->kind = kind;
  plan->bm = kind == 0 ? (!form.fp4 ? 16 : rows <= 8 ? 8 : rows <= 16 || D > 128 ? 16 : 32) : kind == 1 ? 64 : kind == 2 ? 128 : 256;
  plan->bn = kind >= 2 ? kTcBN : form.fp4 ? kFp4BN : kAttnBN;
  plan->rows = rows < 1 ? 1 : rows < plan->bm ? rows : plan->bm;
  plan->dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  int threads = kAttnThreads;
  if (kind >= 2) {
    plan->smem = kind == 2 ? (plan->dp == 64 ? AttnTcGeom<64, false>::kSmem : AttnTcGeom<128, false>::kSmem)
                           : (plan->dp == 64 ? AttnTcGeom<64, true>::kSmem : AttnTcGeom<128, true>::kSmem);
    threads = form.fp4 ? kTcFp4Threads : kTcThreads;
  } else if (form.fp4) {
    plan->smem = attn_fp4_smem(plan->dp, plan->bm);
  } else {
    plan->smem = form.bf16 ? attn_mma_smem<true>(plan->dp, plan->bm) : attn_mma_smem<false>(plan->dp, plan->bm);
  }
  int occ = 0;
  const cudaError_t e = resident(kernel_of(form, *plan), threads, plan->smem, &occ);
  plan->grid = sms * (kind >= 2 ? 1 : occ);   // the tcgen05 kernel takes all of an SM's TMEM
  return e;
}

// The tcgen05 kernel where a request and key head have more than 16 rows, heads are of 64 to 128 values and
// pages are whole TMA boxes; else 16- and 64-row tiles by mma.sync.  Measured, tcgen05 against mma.sync: 64
// requests over caches ragged to 4096 keys, 8 key heads of 128: 16 rows 120 : 113 us, 32 rows 115 : 160, 64
// rows 130 : 188; single tokens (4 rows) to 8192 keys 235 : 195 (a 128-row product for 4 rows, and one warp's
// softmax in the way of every key tile).  Where the tcgen05 kernel has no form, mma.sync is several times slower:
// 32 x 17 tokens, 64/8 heads of 128, ragged to 16384, pages of 24 (1.23 GB) 848, of 64 (1.11 GB) 222 us; 2 x 2048
// tokens behind 14336, 32/8 heads, pages of 24 3535, of 128 667-745 us; the same with 16/4 heads of 256 5177 us.
int attention_kind(int rows, int D, int page_size, float scale) {
  const bool pow2 = (page_size & (page_size - 1)) == 0;
  if (rows > 16 && D >= 64 && D <= 128 && pow2 && page_size >= 8 && scale > 0.f) return rows > 128 ? 3 : 2;
  return rows <= 16 ? 0 : 1;
}

// Over caches in 4 bits: tiles of 8, 16 or 32 rows by mma.sync for up to 32 rows, for negative scales and heads above
// 128 values (16 rows at most there: O fills the registers), else the tcgen05 kernel.  Measured, 64 requests ragged to 8192
// keys, 8 key heads of 128 (332 MB): 4 rows 73 us (in tiles of 16 rows 92, tcgen05 208), 16 rows 111 (224), 20 rows 146 (two
// tiles of 16 176, tcgen05 205), 32 rows 174 (209, 228); by tcgen05 40 rows 227 (two tiles of 32 305), 64 rows 230 (324).
// 8 heads of 64, mma.sync : tcgen05: 16 rows 75 : 181, 32 rows 105 : 185, 40 rows 184 : 192, 64 rows 187 : 181, 96 rows 280 : 194.
// Heads that are not whole pieces (80; 96 alike), which both kernels read in 8-byte steps: 16 rows 156 : 463, 32 rows 218 :
// 462, 40 rows 383 : 428, 64 rows 408 : 462, 96 rows 585 : 458, so there the border could lie at 64 rows (12 %).
int attention_fp4_kind(int rows, int D, float scale) {
  if (rows > 32 && D <= 128 && scale > 0.f) return rows > 128 ? 3 : 2;
  return 0;
}

// cuTensorMapEncodeTiled, looked up once through the runtime (the library does not link the driver).
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A cache [pages, heads, page_size, dim] as TMA sees it; boxes of 64 values x one page (128 tokens at most).
static bool encode_cache(bool bf16, const PagedBatch& c, void* at, long long page, long long token, long long head,
                         CUtensorMap* map) {
  const EncodeFn fn = encode_fn();
  if (!fn || page <= 0 || token <= 0 || head <= 0) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(token) * 2, static_cast<cuuint64_t>(head) * 2,
                                 static_cast<cuuint64_t>(page) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(c.page_size < kTcBN ? c.page_size : kTcBN), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  auto encode = [&] {
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, at, dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  // a driver call, unlike the runtime's, does not give a thread its context: the first call of a thread lacks one
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess) r = encode();
  return r == CUDA_SUCCESS;
}

bool attention_maps(bool bf16, const PagedBatch& c, AttnMaps* maps) {
  static_assert(sizeof(CUtensorMap) == sizeof(maps->k), "a tensor map is 128 bytes");
  return encode_cache(bf16, c, c.k, c.k_page, c.k_token, c.k_head, reinterpret_cast<CUtensorMap*>(maps->k)) &&
         encode_cache(bf16, c, c.v, c.v_page, c.v_token, c.v_head, reinterpret_cast<CUtensorMap*>(maps->v));
}

cudaError_t launch_attention(const AttnForm& form, const AttnPlan& plan, const AttnParams& p, const AttnMaps& maps,
                             cudaStream_t stream) {
  AttnParams copy = p;
  AttnMaps m = maps;
  void* tc[] = {m.k, m.v, &copy};
  void* mma[] = {&copy};
  return cudaLaunchKernel(kernel_of(form, plan), dim3(plan.grid), dim3(plan.kind < 2 ? kAttnThreads : form.fp4 ? kTcFp4Threads : kTcThreads),
                          plan.kind >= 2 ? tc : mma, plan.smem, stream);
}

cudaError_t launch_attention_combine(bool bf16, const AttnPlan& plan, const AttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // A warp a row where an item has as many as it may.  Four rows a warp: 8 tokens of 16/2 heads of 64 over 28745 keys, whose
  // partials of 38 CTAs a row are joined one after the other, 70 us for 31 (in 4 bits 64 for 30), 64 x 8 tokens of 32/8
  // heads of 128 to 4096 keys 130 for 123; prompts and long batches the same.
  cfg.gridDim = dim3(plan.grid, (plan.rows + 3) / 4, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<true>, p, plan.bm)
              : cudaLaunchKernelEx(&cfg, attn_combine_kernel<false>, p, plan.bm);
}

}  // namespace sv
