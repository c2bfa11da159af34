// attn_delta_prep.cu -- the gated delta rule's records: J, P~ and the gates of every chunk.
//
// A CTA makes one record (64 tokens of one value head).  [K; Q] K^T is a product on the tensor cores; thread t
// owns row t of -M, thread 64 + t row t of P, and solves X (1 + B M) = row from the last column to the first,
//     X_s = row_s - sum over i > s of X_i (beta_i M_is),
// against rows of B M that all threads read from shared memory at the same time: 32 columns at a time, with a
// product on the tensor cores between the two halves (rows 32 on; X's later columns times B M's corner, both
// in three terms).
// Bound by these reads, one step behind the other (the same 16 bytes for all of a warp still take four turns
// of shared memory): 88 us for 16384 rows of 16 heads, four CTAs an SM, where the records' 217 MB take 32.
// Both rows in one of 64 threads, each read serving two: 113 us in one piece, 106 in two blocks.
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

constexpr int kPrepThreads = 2 * kDelta;
constexpr int kBlock = kDelta / 2;
// shared memory, from a 1024-byte boundary: panels of 64 rows of K over 64 of Q; in their place afterwards
constexpr int kOffDown = kDelta * kDelta * 4;  // B M; a first operand of 128 rows, whose rows 32 on and 96 on are used
constexpr int kDownTerm = kPrepThreads * kTermRow, kCornerTerm = kBlock * kTermRow;
constexpr int kOffCorner = kOffDown + kTerms * kDownTerm;  // the second operand: B M's corner
constexpr int kPrepBytes = kOffCorner + kTerms * kCornerTerm + 1024;
static_assert(kPrepBytes >= 2 * kPanelBytes + 1024);

struct PrepArgs {
  CUtensorMap mq, mk;
  Gates g, beta;
  const int32_t* cu;
  uint8_t* records;
  int total, nseq, ratio, Hv, K;
};

// X (1 + B M) = row within the columns FIRST to FIRST + 31, from the last to the first: bm[s][i] = beta_i M_is,
// zero for i <= s.
template <int FIRST>
__device__ __forceinline__ void solve(f2 (&x)[kDelta / 2], uint32_t bm) {
#pragma unroll
  for (int s = kBlock - 2; s >= 0; --s) {
    f2 acc[2] = {0, 0};
    // all reads of a step first: one after the other's use, each would wait for its own
    uint4 m[kBlock / 4];
#pragma unroll
    for (int q = kBlock / 4 - 1; q >= (s + 1) / 4; --q) m[q] = lds128_at(bm + ((FIRST + s) * kDelta + FIRST + 4 * q) * 4);
#pragma unroll
    for (int q = kBlock / 4 - 1; q >= (s + 1) / 4; --q) {  // what the last step made comes last
      acc[0] = f2_fma(x[FIRST / 2 + 2 * q], f2_pack(__uint_as_float(m[q].x), __uint_as_float(m[q].y)), acc[0]);
      acc[1] = f2_fma(x[FIRST / 2 + 2 * q + 1], f2_pack(__uint_as_float(m[q].z), __uint_as_float(m[q].w)), acc[1]);
    }
    f2& to = x[(FIRST + s) / 2];
    float a, b, lo, hi;
    cconv::f2_unpack(f2_add(acc[0], acc[1]), a, b);
    cconv::f2_unpack(to, lo, hi);
    to = s % 2 ? f2_pack(lo, hi - (a + b)) : f2_pack(lo - (a + b), hi);
  }
}
__device__ __forceinline__ void unpack_pairs(const f2* x, float* y) {
#pragma unroll
  for (int k = 0; k < 4; ++k) cconv::f2_unpack(x[k], y[2 * k], y[2 * k + 1]);
}

// A row's terms to the record (neighbouring threads have neighbouring rows).
__device__ __forceinline__ void store_row(const f2 (&x)[kDelta / 2], uint8_t* record, int row) {
#pragma unroll
  for (int i = 0; i < kDelta / 8; ++i) {
    uint4 t[kTerms];
    float v[8];
    unpack_pairs(x + 4 * i, v);
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
  __shared__ alignas(8) uint64_t bars[3];
  __shared__ uint32_t tmem_at;
  __shared__ alignas(16) float logs[kDelta], betas[kDelta];  // [s]: log2 of token s + 1's decay
  const uint32_t loaded = smem_addr(bars), done = loaded + 8, joined = done + 8;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    bar_init(loaded, 1);
    bar_init(done, 1);
    bar_init(joined, 1);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_at, kDelta);
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
          const uint64_t kq = tile_desc(smem, 0);
          const uint32_t desc = mma_desc(kDelta, false, false);
          for (int j = 0; j < ksteps; ++j) mma_ss(tmem, kq + col_step(j), kq + col_step(j), desc, j > 0);
        } else {
          drain(loaded, 1);
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
    const int t = tid % kDelta;
    const bool own_p = tid >= kDelta, late = warp % 2;  // a row of P; one of rows 32 on
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    f2 x[kDelta / 2];
    __syncthreads();  // (K and Q are not needed any more)
    {
      const float b = betas[t], sign = own_p ? 1.f : -1.f;
      const int end = t >= n ? 0 : own_p ? t + 1 : t;  // columns of the row that are not zero
      float e = 0.f;  // log2 of the decay from s to t
#pragma unroll
      for (int h = 1; h >= 0; --h) {
        uint32_t y[32];
        tmem_ld32(mine + 32 * h, y);
        tmem_wait_ld();
        tmem_use32(y);
        float below[8];
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const float4 l = *reinterpret_cast<const float4*>(&logs[32 * h + 4 * i]);  // of tokens s + 1
          float m[4];
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            const int s = 32 * h + 4 * i + j;
            if (s < t) e += j == 3 ? l.w : j == 2 ? l.z : j == 1 ? l.y : l.x;
            m[j] = s < end ? __uint_as_float(y[4 * i + j]) * exp2_fast(e) : 0.f;
            below[4 * (i % 2) + j] = b * m[j];
            if (!own_p && (h == 1 || !late)) bm[s * kDelta + t] = b * m[j];
          }
          // (columns 0 to 31 of rows 32 on: a factor of the product below)
          if (h == 0 && warp == 1 && i % 2 == 0) put_terms8(smem + kOffCorner, kCornerTerm, lane, i / 2, below);
          x[16 * h + 2 * i] = f2_pack(sign * m[0], sign * m[1]);
          x[16 * h + 2 * i + 1] = f2_pack(sign * m[2], sign * m[3]);
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    // rows below 32 have zeros in the columns from 32 on; of the others these are solved first, and their
    // product with B M's corner (columns 0 to 31 of rows 32 on) leaves two blocks of one kind
    if (late) {
      solve<kBlock>(x, smem);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[8];
        unpack_pairs(x + kBlock / 2 + 4 * i, v);
        put_terms8(smem + kOffDown, kDownTerm, tid, i, v);
      }
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (warp == 1 && elect_one()) {
        tc_fence_after();
        const uint32_t desc = mma_desc(kBlock, false, true);
        for (int a = 0; a < kTerms; ++a)
          for (int b = 0; a + b < kTerms; ++b)
            for (int j = 0; j < kBlock / 16; ++j)
              mma_ss(tmem, term_desc(smem + kOffDown + a * kDownTerm, 0) + 2 * j,
                     term_desc(smem + kOffCorner + b * kCornerTerm, 0) + j * kTermStep, desc, a + b + j > 0);
        mma_commit(joined);
      }
      __syncwarp();
      ok = wait_phase(joined, 0) && ok;
      tc_fence_after();
      uint32_t y[32];
      tmem_ld32(mine, y);
      tmem_wait_ld();
      tmem_use32(y);
#pragma unroll
      for (int i = 0; i < kBlock / 2; ++i) x[i] = f2_fma(pair(y, i), f2_splat(-1.f), x[i]);
    }
    solve<0>(x, smem);
    store_row(x, record, lane_of(t) + (own_p ? kOther : 0));
    if (!ok) atomicOr(&g_fault_prep, kFaultWait);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, kDelta);
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
