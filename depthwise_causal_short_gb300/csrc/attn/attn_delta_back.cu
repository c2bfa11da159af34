// attn_delta_back.cu -- launches of the chain backwards: behind the chain of the states, or both at once.
#include "attn_delta_back.cuh"
#include "attn_delta_chain.cuh"

namespace cattn {

static __device__ unsigned g_fault_back;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_back, sizeof(*out))) != cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_back, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

__global__ void __launch_bounds__(back::kThreads, 1) cattn_delta_back_kernel(const __grid_constant__ back::Args p) {
  back::run<false>(p, static_cast<int>(blockIdx.x), &g_fault_back);
}

// Both chains: the first half of the CTAs is the chain of the states (a CTA with as many threads as the other
// needs), and none waits for another.
struct BothArgs {
  chain::Args states;
  back::Args back;
  int ctas;  // of each
};
constexpr int kBothBytes = chain::kBytes > back::kBytes ? chain::kBytes : back::kBytes;
static_assert(chain::kThreads <= back::kThreads);
__global__ void __launch_bounds__(back::kThreads, 1) cattn_delta_both_kernel(const __grid_constant__ BothArgs p) {
  const int cta = static_cast<int>(blockIdx.x);
  if (cta < p.ctas)
    chain::run<true>(p.states, cta, &g_fault_back);
  else
    back::run<true>(p.back, cta - p.ctas, &g_fault_back);
}

// Behind both: dbeta = du . z, and <S_0, D_0> at the anchors.  A CTA for each chunk and value head, a warp in the
// place of each row warp.
struct JoinArgs {
  const int32_t* cu;
  const float *z, *du, *anchors, *danchors;
  float *bdots, *adots;
  int total, nseq, Hv, tiles;
};
__global__ void __launch_bounds__(kRowWarps * 32) cattn_delta_join_kernel(const JoinArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int place = threadIdx.x / 32, lane = threadIdx.x % 32, hv = static_cast<int>(blockIdx.x % p.Hv);
  const int64_t slot = blockIdx.x / p.Hv;
  Chunk x;
  if (!find_chunk(p.cu, p.nseq, p.total, slot, lane, x)) return;
  const int quarter = place % 4, h = place / 4, row = quarter * 32 + lane, t = quarter * 16 + lane / 4;
  const bool anchor = x.c > 0 && x.c % kAnchorChunks == 0;
#pragma unroll 2
  for (int tile = 0; tile < p.tiles; ++tile) {
    const int64_t from = pairs_at((slot * p.Hv + hv) * p.tiles + tile, place, lane);
    const ulonglong2 *z = reinterpret_cast<const ulonglong2*>(p.z + from), *du = reinterpret_cast<const ulonglong2*>(p.du + from);
    const ulonglong2 z0 = z[0], z1 = z[kPairsNext], du0 = du[0], du1 = du[kPairsNext];
    const f2 sums[2] = {f2_fma(z0.x, du0.x, f2_mul(z1.x, du1.x)), f2_fma(z0.y, du0.y, f2_mul(z1.y, du1.y))};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float a, b;
      cconv::f2_unpack(sums[r], a, b);
      float du_z = a + b;
      du_z += __shfl_xor_sync(0xffffffffu, du_z, 1);
      du_z += __shfl_xor_sync(0xffffffffu, du_z, 2);
      if (t + 8 * r < x.n && (lane & 3) == 0)
        p.bdots[(static_cast<int64_t>(tile * 2 + h) * p.Hv + hv) * p.total + x.row0 + t + 8 * r] = du_z;
    }
    if (anchor) {
      const int64_t at = (anchor_of(x.a, x.c) * p.Hv + hv) * p.tiles + tile;
      const int64_t first = at * kAnchorFloats + row * kColumns + h * 16;
      const float4 *s = reinterpret_cast<const float4*>(p.anchors + first);
      const float4 *d = reinterpret_cast<const float4*>(p.danchors + first);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += dot4(d[j], s[j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) p.adots[at * kRowWarps + place] = sum;
    }
  }
}

int launch_delta_back(const DeltaCall& c, cudaStream_t stream) {
  back::Args a{};
  const int rc = back::args_of(c, a);
  if (rc != CCONV_OK) return rc;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_delta_back_kernel), back::kBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(cattn_delta_back_kernel, dim3(chain::ctas(c)), dim3(back::kThreads), back::kBytes, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_delta_both(const DeltaCall& c, cudaStream_t stream) {
  BothArgs a{};
  int rc = chain::args_of(c, a.states);
  if (rc == CCONV_OK) rc = back::args_of(c, a.back);
  if (rc != CCONV_OK) return rc;
  a.ctas = chain::ctas(c);
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_delta_both_kernel), kBothBytes) != CCONV_OK ||
      launch_pdl(cattn_delta_both_kernel, dim3(2 * a.ctas), dim3(back::kThreads), kBothBytes, stream, a) != cudaSuccess)
    return CCONV_ERR_CUDA;
  const JoinArgs j{c.cu, c.z, c.du, c.anchors, c.danchors, c.bdots, c.adots, c.s.total, c.s.nseq, c.s.Hv, delta_tiles(c.s.V)};
  const int64_t chunks = delta_slots(c.s.total, c.s.nseq) * c.s.Hv;
  return launch_pdl(cattn_delta_join_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kRowWarps * 32), 0, stream, j) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cattn
