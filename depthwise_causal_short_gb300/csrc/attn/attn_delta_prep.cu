// attn_delta_prep.cu -- the gated delta rule's records: J, P~ and the gates of every chunk.
//
// A CTA makes one record (64 tokens of one value head).  [K; Q] K^T is one product of 128 x 64 on
// the tensor cores; thread r then owns row r of [-M; P] and solves X (1 + B M) = row from the last
// column to the first,
//     X_s = row_s - sum over i > s of X_i (beta_i M_is),
// against rows of B M that all threads read from shared memory at the same time.
// Bound by that solve (2016 multiply-adds a thread, as 1008 packed ones).
#include <cudaTypedefs.h>

#include "attn_chunk_host.h"
#include "attn_delta.cuh"

namespace cattn {

static __device__ unsigned g_fault_prep;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_prep, sizeof(*out))) != cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_prep, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

constexpr int kPrepThreads = 128;
// shared memory, from a 1024-byte boundary: the record (K and Q in its place first), then B M
constexpr int kPrepBm = (kRecordBytes + 1023) / 1024 * 1024;
constexpr int kPrepBytes = kPrepBm + kDelta * kDelta * 4 + 1024;
static_assert(2 * 2 * kSideBytes <= kTerms * kJpTerm, "K and Q fit the record's place");

struct PrepArgs {
  CUtensorMap mq, mk;
  Gates g, beta;
  const int32_t* cu;
  uint8_t* records;
  int total, nseq, ratio, Hv, K;
};

__global__ void __launch_bounds__(kPrepThreads) cattn_delta_prep_kernel(const __grid_constant__ PrepArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  float* gates = reinterpret_cast<float*>(base + kTerms * kJpTerm);
  float* bm = reinterpret_cast<float*>(base + kPrepBm);  // [s][i] = beta_i M_is
  __shared__ alignas(8) uint64_t bars[2];
  __shared__ uint32_t tmem_at;
  __shared__ float logs[kDelta];  // log2 of the tokens' decays
  const uint32_t loaded = smem_addr(bars), done = loaded + 8;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    bar_init(loaded, 1);
    bar_init(done, 1);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_at, 64);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int hv = static_cast<int>(blockIdx.x % p.Hv);
  const int64_t slot = blockIdx.x / p.Hv;
  int row0 = 0, n = 0;
  const bool live = find_chunk(p.cu, p.nseq, p.total, slot, lane, row0, n);
  bool ok = true;
  if (live) {
    const int panels = p.K > kPanelCols ? 2 : 1, ksteps = (p.K + 15) / 16;
    if (warp == 0) {
      if (elect_one()) {
        bar_expect(loaded, panels * 2 * kSideBytes);
        for (int c = 0; c < panels; ++c) {
          load_box(smem + c * kPanelBytes, &p.mk, loaded, c * kPanelCols, hv / p.ratio, row0);
          load_box(smem + c * kPanelBytes + kSideBytes, &p.mq, loaded, c * kPanelCols, hv / p.ratio, row0);
        }
        ok = wait_phase(loaded, 0);
        if (ok) {
          const uint64_t d = tile_desc(smem, 0);
          const uint32_t desc = mma_desc(kDelta, false, false);
          for (int j = 0; j < ksteps; ++j) mma_ss(tmem, d + col_step(j), d + col_step(j), desc, j > 0);
        }
        mma_commit(done);
      }
      __syncwarp();
    } else if (warp == 1) {
      // gates: two tokens a lane; sums of one sign from the front and from the back
      float g[2], b[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 2 * lane + j;
        g[j] = t < n ? kLog2e * p.g.at(row0 + t, hv) : 0.f;
        b[j] = t < n ? __ldg(p.beta.p + (row0 + t) * p.beta.st + hv * p.beta.sh) : 0.f;
      }
      float up = g[0] + g[1], down = up;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, up, o), y = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up += x;
        if (lane + o < 32) down += y;
      }
      float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
      if (lane == 0) before = 0.f;
      if (lane == 31) after = 0.f;
      const int t = 2 * lane;
      logs[t] = g[0], logs[t + 1] = g[1];
      gates[kEf + t] = exp2_fast(before + g[0]), gates[kEf + t + 1] = exp2_fast(before + g[0] + g[1]);
      gates[kEb + t] = exp2_fast(g[1] + after), gates[kEb + t + 1] = exp2_fast(after);
      gates[kBeta + t] = b[0], gates[kBeta + t + 1] = b[1];
      const float all = __shfl_sync(0xffffffffu, down, 0);
      gates[kTotal + t] = exp2_fast(all), gates[kTotal + t + 1] = 0.f;
    }
    __syncthreads();
    ok = wait_phase(done, 0) && ok;
    tc_fence_after();
    // thread r: row r of [-M; P]
    const int t = tid & (kDelta - 1);
    const bool side = tid >= kDelta;
    float x[kDelta];
    {
      uint32_t y[2][32];
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16), y[0]);
      tmem_ld32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + 32, y[1]);
      tmem_wait_ld();
      tmem_use32(y[0]);
      tmem_use32(y[1]);
      float e = 0.f;  // log2 of the decay from s to t
#pragma unroll
      for (int s = kDelta - 1; s >= 0; --s) {
        if (s < t) e += logs[s + 1 < kDelta ? s + 1 : s];
        const float v = __uint_as_float(y[s / 32][s % 32]) * exp2_fast(e);
        x[s] = t < n && (s < t || (s == t && side)) ? (side ? v : -v) : 0.f;
      }
    }
    if (!side) {
      const float b = -gates[kBeta + t];
#pragma unroll
      for (int s = 0; s < kDelta; ++s) bm[s * kDelta + t] = b * x[s];
    }
    tc_fence_before();
    __syncthreads();
#pragma unroll
    for (int s = kDelta - 2; s >= 0; --s) {
      f2 acc[2] = {0, 0};
#pragma unroll
      for (int q = (s + 1) / 4; q < kDelta / 4; ++q) {
        const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(bm + s * kDelta + 4 * q);
        // (columns up to s hold zeros)
        acc[0] = f2_fma(f2_pack(x[4 * q], x[4 * q + 1]), m.x, acc[0]);
        acc[1] = f2_fma(f2_pack(x[4 * q + 2], x[4 * q + 3]), m.y, acc[1]);
      }
      float a, b;
      cconv::f2_unpack(f2_add(acc[0], acc[1]), a, b);
      x[s] -= a + b;
    }
#pragma unroll
    for (int j = 0; j < kDelta / 8; ++j) {
      uint4 terms[kTerms];
      split8(x + 8 * j, terms);
      const uint32_t at = smem + swizzled(tid, j);
#pragma unroll
      for (int i = 0; i < kTerms; ++i) sts128(at + i * kJpTerm, terms[i].x, terms[i].y, terms[i].z, terms[i].w);
    }
    cconv::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store(p.records + (slot * p.Hv + hv) * kRecordBytes, smem, kRecordBytes);
      stores_commit();
      stores_wait();
      if (!ok) atomicOr(&g_fault_prep, kFaultWait);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 64);
  }
}

int launch_delta_prep(const DeltaCall& c, cudaStream_t stream) {
  PrepArgs a{};
  int rc = bind_context();
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc != CCONV_OK) return rc;
  a.g = c.g, a.beta = c.beta;
  a.cu = c.cu;
  a.records = c.records;
  a.total = c.s.total, a.nseq = c.s.nseq, a.ratio = c.s.Hv / c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K;
  const int64_t ctas = delta_slots(c.s.total, c.s.nseq) * c.s.Hv;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_delta_prep_kernel), kPrepBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(cattn_delta_prep_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPrepThreads), kPrepBytes,
                    stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cattn
