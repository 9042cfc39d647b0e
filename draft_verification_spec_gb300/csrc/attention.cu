// Host side of the paged attention (kernel choice, launches) and the kernel that joins items split
// over several CTAs.
#include <map>
#include <mutex>
#include <tuple>

#include "attention_tc.cuh"

namespace sv {

template <>
const void* attn_mma_fn<true>(int dp, int bm);
template <>
const void* attn_mma_fn<false>(int dp, int bm);
template <>
const void* attn_tc_fn<true>(int dp, bool wide);
template <>
const void* attn_tc_fn<false>(int dp, bool wide);

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
#pragma unroll 4
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
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int tok = attn_token(p, j.row0 + r);
    const long long row = static_cast<long long>(j.token0 + tok) * p.Hq + j.head0 + (j.row0 + r - tok * p.G);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = lane * 4 + i * 128;
      if (d < D)
        *reinterpret_cast<uint2*>(p.out + (row * D + d) * 2) =
            make_uint2(A::pack(acc[i].x * inv, acc[i].y * inv), A::pack(acc[i].z * inv, acc[i].w * inv));
    }
    if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : ninf();
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

static const void* kernel_of(bool bf16, const AttnPlan& plan) {
  if (plan.kind >= 2) return bf16 ? attn_tc_fn<true>(plan.dp, plan.kind == 3) : attn_tc_fn<false>(plan.dp, plan.kind == 3);
  return bf16 ? attn_mma_fn<true>(plan.dp, plan.bm) : attn_mma_fn<false>(plan.dp, plan.bm);
}

cudaError_t attention_plan(bool bf16, int kind, int rows, int D, int sms, AttnPlan* plan) {
  plan->kind = kind;
  plan->bm = kind == 0 ? 16 : kind == 1 ? 64 : kind == 2 ? 128 : 256;
  plan->bn = kind >= 2 ? kTcBN : kAttnBN;
  plan->rows = rows < 1 ? 1 : rows < plan->bm ? rows : plan->bm;
  plan->dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  int threads = kAttnThreads;
  if (kind >= 2) {
    plan->smem = kind == 2 ? (plan->dp == 64 ? AttnTcGeom<64, false>::kSmem : AttnTcGeom<128, false>::kSmem)
                           : (plan->dp == 64 ? AttnTcGeom<64, true>::kSmem : AttnTcGeom<128, true>::kSmem);
    threads = kTcThreads;
  } else {
    plan->smem = bf16 ? attn_mma_smem<true>(plan->dp, plan->bm) : attn_mma_smem<false>(plan->dp, plan->bm);
  }
  int occ = 0;
  const cudaError_t e = resident(kernel_of(bf16, *plan), threads, plan->smem, &occ);
  plan->grid = sms * (kind >= 2 ? 1 : occ);   // the tcgen05 kernel takes all of an SM's TMEM
  return e;
}

// The tcgen05 kernel where a request and key head have more than 16 rows, heads are of 64 to 128 values and
// pages are whole TMA boxes; else 16- and 64-row tiles by mma.sync.  Measured, tcgen05 against mma.sync: 64
// requests over caches ragged to 4096 keys, 8 key heads of 128: 16 rows 120 : 113 us, 32 rows 115 : 160, 64
// rows 130 : 188; single tokens (4 rows) to 8192 keys 235 : 195 (a 128-row product for 4 rows, and one warp's
// softmax in the way of every key tile).  Where the tcgen05 kernel has no form, mma.sync is several times slower:
// 32 x 17 tokens, 64/8 heads of 128, ragged to 16384, pages of 24 (1.23 GB) 848, of 64 (1.11 GB) 222 us; 2 x 2048
// tokens behind 14336, 32/8 heads, pages of 24 3535, of 128 750 us; the same with 16/4 heads of 256 5177 us.
int attention_kind(int rows, int D, int page_size, float scale) {
  const bool pow2 = (page_size & (page_size - 1)) == 0;
  if (rows > 16 && D >= 64 && D <= 128 && pow2 && page_size >= 8 && scale > 0.f) return rows > 128 ? 3 : 2;
  return rows <= 16 ? 0 : 1;
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

cudaError_t launch_attention(bool bf16, const AttnPlan& plan, const AttnParams& p, const AttnMaps& maps, cudaStream_t stream) {
  AttnParams copy = p;
  AttnMaps m = maps;
  void* tc[] = {m.k, m.v, &copy};
  void* mma[] = {&copy};
  return cudaLaunchKernel(kernel_of(bf16, plan), dim3(plan.grid), dim3(plan.kind >= 2 ? kTcThreads : kAttnThreads),
                          plan.kind >= 2 ? tc : mma, plan.smem, stream);
}

cudaError_t launch_attention_combine(bool bf16, const AttnPlan& plan, const AttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // four rows a warp where an item has as many as it may, a warp a row in 16-row tiles
  cfg.gridDim = dim3(plan.grid, plan.bm <= 16 ? 4 : (plan.rows + 15) / 16, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<true>, p, plan.bm)
              : cudaLaunchKernelEx(&cfg, attn_combine_kernel<false>, p, plan.bm);
}

}  // namespace sv
