// Host side of the paged attention (kernel choice, launches) and the kernel that joins items split
// over several CTAs.
#include <map>
#include <mutex>
#include <tuple>

#include "attention_mma.cuh"

namespace sv {

template <>
const void* attn_mma_fn<true>(int dp, int bm);
template <>
const void* attn_mma_fn<false>(int dp, int bm);

// One warp per row of the item that begins in CTA blockIdx.x's run and goes on in others': the
// partials in key order, each scaled by 2^(its maximum - the largest).  fp32.
template <int BN, int DTYPE>
__global__ void __launch_bounds__(128) attn_combine_kernel(const AttnParams p, int bm) {
  __shared__ AttnSchedSmem<128> sched;
  const AttnSplit split = attn_split<BN>(p, bm, sched);
  const int c1 = blockIdx.x;
  if (c1 + 1 >= split.n) return;
  const long long u0 = split.begin(c1), u1 = split.begin(c1 + 1);
  const AttnCursor cur = attn_locate<BN>(p, bm, u1 - 1, sched);
  const long long start = u1 - 1 - cur.at, end = start + cur.count;
  if (start < u0 || end <= u1) return;
  const int c2 = split.owner(end - 1);
  const int r0 = cur.t * bm, rows = min(cur.req.nq * p.G - r0, bm);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, D = p.c.D;
  for (int r = blockIdx.y * 4 + threadIdx.x / 32; r < rows; r += gridDim.y * 4) {
    auto slot = [&](int c) { return static_cast<long long>(c == c1 && start != u0 ? 2 * c + 1 : 2 * c) * bm + r; };
    float m = ninf();
    for (int c = c1 + lane; c <= c2; c += 32) m = fmaxf(m, __ldcg(p.part_ml + slot(c) * 2));
    m = warp_maxf(m);
    const float ref = m == ninf() ? 0.f : m;
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    float l = 0.f;
#pragma unroll 4
    for (int c = c1; c <= c2; ++c) {
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
    const long long row = static_cast<long long>(cur.req.q0 + (r0 + r) / p.G) * p.Hq + cur.h * p.G + (r0 + r) % p.G;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int d = lane * 4 + i * 128;
      if (d < D) {
        using A = AttnType<DTYPE == 1>;
        *reinterpret_cast<uint2*>(p.out + (row * D + d) * 2) =
            make_uint2(A::pack(acc[i].x * inv, acc[i].y * inv), A::pack(acc[i].z * inv, acc[i].w * inv));
      }
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

cudaError_t attention_mma_plan(bool bf16, int rows, int D, int sms, AttnPlan* plan) {
  plan->kind = rows <= 16 ? 0 : 1;
  plan->bm = rows <= 16 ? 16 : 64;
  plan->bn = kAttnBN;
  plan->dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  plan->smem = bf16 ? attn_mma_smem<true>(plan->dp, plan->bm) : attn_mma_smem<false>(plan->dp, plan->bm);
  const void* fn = bf16 ? attn_mma_fn<true>(plan->dp, plan->bm) : attn_mma_fn<false>(plan->dp, plan->bm);
  int occ = 0;
  const cudaError_t e = resident(fn, kAttnThreads, plan->smem, &occ);
  plan->grid = sms * occ;
  return e;
}

cudaError_t launch_attention_mma(bool bf16, const AttnPlan& plan, const AttnParams& p, cudaStream_t stream) {
  const void* fn = bf16 ? attn_mma_fn<true>(plan.dp, plan.bm) : attn_mma_fn<false>(plan.dp, plan.bm);
  AttnParams copy = p;
  void* args[] = {&copy};
  return cudaLaunchKernel(fn, dim3(plan.grid), dim3(kAttnThreads), args, plan.smem, stream);
}

cudaError_t launch_attention_combine(int dtype, const AttnPlan& plan, const AttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(plan.grid, plan.bm <= 16 ? 4 : 16, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (plan.bn == 64)
    return dtype == 1 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<64, 1>, p, plan.bm)
                      : cudaLaunchKernelEx(&cfg, attn_combine_kernel<64, 2>, p, plan.bm);
  return dtype == 1 ? cudaLaunchKernelEx(&cfg, attn_combine_kernel<128, 1>, p, plan.bm)
                    : cudaLaunchKernelEx(&cfg, attn_combine_kernel<128, 2>, p, plan.bm);
}

}  // namespace sv
