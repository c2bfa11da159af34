// attn_delta_prep.cu -- the gated delta rule's records: J, P~ and the gates of every chunk.
//
// A CTA makes one record (64 tokens of one value head).  K K^T and Q K^T are products on the tensor
// cores; thread t then owns row t of -M and of P and solves X (1 + B M) = row from the last column to the
// first,
//     X_s = row_s - sum over i > s of X_i (beta_i M_is),
// against rows of B M that all threads read from shared memory at the same time.
// Bound by these reads: the same 16 bytes for all of a warp still take four turns of shared memory.  So
// each read serves two rows, and the warp of the first 32 tokens leaves out what is zero.
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

constexpr int kPrepThreads = 64;
// shared memory, from a 1024-byte boundary: panels of 64 rows of K over 64 of Q (and what the product
// with Q reads behind them); B M in their place afterwards
constexpr int kPrepBytes = 2 * kPanelBytes + kSideBytes + 1024;

struct PrepArgs {
  CUtensorMap mq, mk;
  Gates g, beta;
  const int32_t* cu;
  uint8_t* records;
  int total, nseq, ratio, Hv, K;
};

// X (1 + B M) = rows, from the last of N columns to the first, for two rows at once (a row of B M in
// shared memory serves both): bm[s][i] = beta_i M_is, zero for i <= s.
template <int N>
__device__ __forceinline__ void solve(f2 (&x)[2][kDelta / 2], uint32_t bm) {
#pragma unroll
  for (int s = N - 2; s >= 0; --s) {
    f2 acc[2][2] = {{0, 0}, {0, 0}};
    // all reads of a step first: one after the other's use, each would wait for its own
    uint4 m[N / 4];
#pragma unroll
    for (int q = N / 4 - 1; q >= (s + 1) / 4; --q) m[q] = lds128_at(bm + (s * kDelta + 4 * q) * 4);
#pragma unroll
    for (int q = N / 4 - 1; q >= (s + 1) / 4; --q) {  // what the last step made comes last
      const f2 lo = f2_pack(__uint_as_float(m[q].x), __uint_as_float(m[q].y));
      const f2 hi = f2_pack(__uint_as_float(m[q].z), __uint_as_float(m[q].w));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        acc[r][0] = f2_fma(x[r][2 * q], lo, acc[r][0]);
        acc[r][1] = f2_fma(x[r][2 * q + 1], hi, acc[r][1]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float a, b, lo, hi;
      cconv::f2_unpack(f2_add(acc[r][0], acc[r][1]), a, b);
      cconv::f2_unpack(x[r][s / 2], lo, hi);
      x[r][s / 2] = s % 2 ? f2_pack(lo, hi - (a + b)) : f2_pack(lo - (a + b), hi);
    }
  }
}

// A row's three terms to the record (neighbouring threads have neighbouring rows).
__device__ __forceinline__ void store_row(const f2 (&x)[kDelta / 2], uint8_t* record, int row) {
#pragma unroll
  for (int i = 0; i < kDelta / 8; ++i) {
    uint4 t[kTerms];
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) cconv::f2_unpack(x[4 * i + k], v[2 * k], v[2 * k + 1]);
    split8(v, t);
#pragma unroll
    for (int s = 0; s < kTerms; ++s) *reinterpret_cast<uint4*>(record + record_piece(s, i, row)) = t[s];
  }
}

__global__ void __launch_bounds__(kPrepThreads, 4) cattn_delta_prep_kernel(const __grid_constant__ PrepArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  float* bm = reinterpret_cast<float*>(base);  // [s][i] = beta_i M_is
  __shared__ alignas(8) uint64_t bars[2];
  __shared__ uint32_t tmem_at;
  __shared__ alignas(16) float logs[kDelta], betas[kDelta];  // [s]: log2 of token s + 1's decay
  const uint32_t loaded = smem_addr(bars), done = loaded + 8;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    bar_init(loaded, 1);
    bar_init(done, 1);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_at, 128);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int hv = static_cast<int>(blockIdx.x % p.Hv);
  const int64_t slot = blockIdx.x / p.Hv;
  Chunk chunk;
  const bool live = find_chunk(p.cu, p.nseq, p.total, slot, lane, chunk);
  const int row0 = live ? chunk.row0 : 0, n = live ? chunk.n : 0;
  bool ok = true;
  if (live) {
    uint8_t* record = p.records + (slot * p.Hv + hv) * kRecordBytes;
    if (warp == 0) {
      if (elect_one()) {
        const int panels = p.K > kPanelCols ? 2 : 1, ksteps = (p.K + 15) / 16;
        bar_expect(loaded, panels * 2 * kSideBytes);
        for (int c = 0; c < panels; ++c) {
          load_box(smem + c * kPanelBytes, &p.mk, loaded, c * kPanelCols, hv / p.ratio, row0);
          load_box(smem + c * kPanelBytes + kSideBytes, &p.mq, loaded, c * kPanelCols, hv / p.ratio, row0);
        }
        ok = wait_phase(loaded, 0);
        if (ok) {
          // lanes 0 to 63 of the results: K K^T in columns 0 to 63, Q K^T in 64 to 127 (M = 128: lanes 64
          // to 127 hold what follows in shared memory, and are not read)
          const uint64_t k = tile_desc(smem, 0), q = tile_desc(smem + kSideBytes, 0);
          const uint32_t desc = mma_desc(kDelta, false, false);
          for (int j = 0; j < ksteps; ++j) {
            mma_ss(tmem, k + col_step(j), k + col_step(j), desc, j > 0);
            mma_ss(tmem + kDelta, q + col_step(j), k + col_step(j), desc, j > 0);
          }
        } else {
          drain(loaded, 1);
        }
        mma_commit(done);
      }
      __syncwarp();
    } else {
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
      if (t > 0) logs[t - 1] = g[0];
      logs[t] = g[1];
      if (lane == 31) logs[t + 1] = 0.f;
      betas[t] = b[0], betas[t + 1] = b[1];
      float2* gates = reinterpret_cast<float2*>(record + kRecordGates) + lane;
      gates[kEf / 2] = make_float2(exp2_fast(before + g[0]), exp2_fast(before + g[0] + g[1]));
      gates[kEb / 2] = make_float2(exp2_fast(g[1] + after), exp2_fast(after));
      gates[kBeta / 2] = make_float2(b[0], b[1]);
      gates[kTotal / 2] = make_float2(exp2_fast(__shfl_sync(0xffffffffu, down, 0)), 0.f);
    }
    __syncthreads();
    ok = wait_phase(done, 0) && ok;
    tc_fence_after();
    // thread t: rows t of -M and of P
    const int t = tid;
    f2 x[2][kDelta / 2];
    __syncthreads();  // (K and Q are not needed any more: B M takes their place)
    {
      const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      const float b = betas[t];
      float e = 0.f;  // log2 of the decay from s to t
#pragma unroll
      for (int h = 1; h >= 0; --h) {
        uint32_t y[2][32];
        tmem_ld32(mine + 32 * h, y[0]);
        tmem_ld32(mine + kDelta + 32 * h, y[1]);
        tmem_wait_ld();
        tmem_use32(y[0]);
        tmem_use32(y[1]);
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const float4 l = *reinterpret_cast<const float4*>(&logs[32 * h + 4 * i]);  // of tokens s + 1
          float m[4], q[4];
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            const int s = 32 * h + 4 * i + j;
            if (s < t) e += j == 3 ? l.w : j == 2 ? l.z : j == 1 ? l.y : l.x;
            const float w = exp2_fast(e);
            m[j] = t < n && s < t ? __uint_as_float(y[0][4 * i + j]) * w : 0.f;
            q[j] = t < n && s <= t ? __uint_as_float(y[1][4 * i + j]) * w : 0.f;
            bm[s * kDelta + t] = b * m[j];
          }
          x[0][16 * h + 2 * i] = f2_pack(-m[0], -m[1]);
          x[0][16 * h + 2 * i + 1] = f2_pack(-m[2], -m[3]);
          x[1][16 * h + 2 * i] = f2_pack(q[0], q[1]);
          x[1][16 * h + 2 * i + 1] = f2_pack(q[2], q[3]);
        }
      }
    }
    __syncthreads();
    // rows below 32 have zeros in the columns from 32 on
    if (warp == 0)
      solve<kDelta / 2>(x, smem);
    else
      solve<kDelta>(x, smem);
    store_row(x[0], record, lane_of(t));
    store_row(x[1], record, lane_of(t) + kOther);
    if (!ok) atomicOr(&g_fault_prep, kFaultWait);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 128);
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
