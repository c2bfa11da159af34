// attn_delta_back.cu -- the gated delta rule's chain backwards: the gradient of the state.
//
// The CTAs, ring, terms and roles of attn_delta_chain.cu, from a sequence's last chunk to its first.
// D, the gradient of the state at the chunk's end, is kept as S is there.  A chunk's products:
//   K D                                -> r' = eb . (K D),  X = beta r'
//   J^T X;  P~^T do                    -> du = r' + J^T X + scale P~^T do,  dv = beta du
//   K^T (-ef . dv);  Q^T (scale ef . do)  -> D = total D + ..
// J and P~ are read from their records with the rows as the contraction.  The products that have do in
// them wait for nothing of the chain; the rows of Q in the first one are not used.
// It leaves dv, the first term of every D, dbeta = du . z and v . dv.
#include <cudaTypedefs.h>

#include "attn_chunk_host.h"
#include "attn_delta.cuh"

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

// shared memory, from a 1024-byte boundary
constexpr int kOffD = kStages * kStageBytes;
constexpr int kOffDx = kOffD + kTerms * kStatePanel;      // X, then -ef . dv
constexpr int kOffDo = kOffDx + kTerms * kTokenPanel;     // scale ef . do
constexpr int kOffDoRaw = kOffDo + kTerms * kTokenPanel;  // do
constexpr int kOffBackBars = kOffDoRaw + kTokenPanel;
constexpr int kBackBytes = kOffBackBars + 16 * 8 + 1024;
static_assert(kBackBytes <= 232448, "shared memory of one CTA");

struct BackArgs {
  CUtensorMap mq, mk;
  Rows v, d_o;
  const int32_t* cu;
  const uint8_t* records;
  const float* z;
  uint8_t* ends;          // [slots][Hv][tiles] first terms of D
  float *vdots, *bdots;   // [2 tiles][Hv][total]
  uint16_t* dv;
  float* dinit;
  float scale;
  int total, nseq, ratio, Hv, K, V, tiles;
};

__global__ void __launch_bounds__(kChainThreads, 1) cattn_delta_back_kernel(const __grid_constant__ BackArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t full = smem + kOffBackBars, empty = full + 8 * kStages;
  const uint32_t dready = empty + 8 * kStages, xready = dready + 8, uready = xready + 8, oready = uready + 8;
  const uint32_t acc1 = oready + 8, acc2 = acc1 + 8, acc3 = acc2 + 8, alldone = acc3 + 8, kept = alldone + 8;
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1 + kRowWarps);
    }
    bar_init(dready, kRowWarps);
    bar_init(xready, kRowWarps / 2);
    bar_init(uready, kRowWarps / 2);
    bar_init(oready, kRowWarps / 2);
    bar_init(acc1, 1);
    bar_init(acc2, 1);
    bar_init(acc3, 1);
    bar_init(alldone, 1);
    bar_init(kept, 1);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_at, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at, tmem2 = tmem + 128;
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int tile = static_cast<int>(blockIdx.x % p.tiles);
  const int hv = static_cast<int>(blockIdx.x / p.tiles % p.Hv);
  const int seq = static_cast<int>(blockIdx.x / p.tiles / p.Hv);
  int row_a, row_b;
  sequence_rows(p.cu, seq, p.total, row_a, row_b);
  if (p.cu[seq] < 0 || p.cu[seq + 1] < p.cu[seq] || p.cu[seq + 1] > p.total) row_b = row_a;  // (reported already)
  const int chunks = (row_b - row_a + kDelta - 1) / kDelta;
  const int64_t slot0 = row_a / kDelta + seq;
  const int col0 = tile * kColumns;
  bool ok = true;

  if (warp == 0) {
    // ---- tiles and records ----
    if (elect_one()) {
      const int panels = p.K > kPanelCols ? 2 : 1, hk = hv / p.ratio;
      int i = 0;
      for (; i < chunks && ok; ++i) {
        const int st = i % kStages, c = chunks - 1 - i;
        if (i >= kStages && !(ok = DELTA_WAIT(empty + 8 * st, i / kStages - 1))) break;
        const uint32_t at = smem + st * kStageBytes, bar = full + 8 * st;
        bar_expect(bar, panels * 2 * kSideBytes + kRecordBytes);
#pragma unroll 1
        for (int j = 0; j < panels; ++j) {
          load_box(at + j * kPanelBytes, &p.mk, bar, j * kPanelCols, hk, row_a + c * kDelta);
          load_box(at + j * kPanelBytes + kSideBytes, &p.mq, bar, j * kPanelCols, hk, row_a + c * kDelta);
        }
        bulk_load(at + kStageKq, p.records + ((slot0 + c) * p.Hv + hv) * kRecordBytes, kRecordBytes, bar);
      }
      for (int st = 0; st < kStages; ++st) drain(full + 8 * st, (i - st + kStages - 1) / kStages);
    }
  } else if (warp == 1) {
    // ---- products ----
    if (elect_one()) {
      const int ksteps = (p.K + 15) / 16;
      const uint64_t dd = term_desc(smem + kOffD, kStatePanel), dx = term_desc(smem + kOffDx, kTokenPanel);
      const uint64_t dos = term_desc(smem + kOffDo, kTokenPanel), raw_do = term_desc(smem + kOffDoRaw, kTokenPanel);
      for (int i = 0; i < chunks && ok; ++i) {
        const int st = i % kStages;
        const uint32_t at = smem + st * kStageBytes;
        if (!(ok = DELTA_WAIT(full + 8 * st, i / kStages))) break;
        if (!(ok = DELTA_WAIT(dready, i))) break;
        tc_fence_after();
        const uint64_t dkq = tile_desc(at, 0);
        const uint32_t wide = mma_desc(3 * kColumns, false, true);
#pragma unroll 1
        for (int j = 0; j < ksteps; ++j) mma_ss(tmem, dkq + col_step(j), dd + j * kTermStep, wide, j > 0);
        mma_commit(acc1);
        if (!(ok = DELTA_WAIT(oready, i))) break;
        tc_fence_after();
        // (M = 128 with 64 columns of A: rows 64 to 127 of the results, made of the next term's
        // bytes, are not read)
        const uint32_t narrow = mma_desc(kColumns, true, true);
#pragma unroll 1
        for (int s = 0; s < kTerms; ++s) {
          const uint64_t da = tile_desc(at + kStageKq + s * kJpTerm + kSideBytes, kJpTerm);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem2 + 3 * kColumns, da + j * kRowStep, raw_do + j * kTermStep, narrow, s + j > 0);
        }
        if (!(ok = DELTA_WAIT(xready, i))) break;
        tc_fence_after();
#pragma unroll 1
        for (int s = 0; s < kTerms; ++s) {
          const uint64_t da = tile_desc(at + kStageKq + s * kJpTerm, kJpTerm);
          const uint32_t desc = mma_desc((kTerms - s) * kColumns, true, true);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem2, da + j * kRowStep, dx + j * kTermStep, desc, s + j > 0);
        }
        mma_commit(acc2);
        const bool more = i + 1 < chunks || p.dinit;
        const uint32_t desc = mma_desc(3 * kColumns, true, true);
        if (more) {
          // (acc1's results were read before xready)
          const uint64_t da = tile_desc(at + kSideBytes, kPanelBytes);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j) mma_ss(tmem, da + j * kRowStep, dos + j * kTermStep, desc, j > 0);
        }
        if (!(ok = DELTA_WAIT(uready, i))) break;
        tc_fence_after();
        if (more) {
          const uint64_t da = tile_desc(at, kPanelBytes);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j) mma_ss(tmem, da + j * kRowStep, dx + j * kTermStep, desc, true);
          mma_commit(acc3);
        }
        mma_commit(empty + 8 * st);
      }
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (warp == 2) {
    // ---- the first term of every D ----
    if (elect_one()) {
      for (int i = 0; i < chunks && ok; ++i) {
        if (!(ok = DELTA_WAIT(dready, i))) break;
        bulk_store(p.ends + (((slot0 + chunks - 1 - i) * p.Hv + hv) * p.tiles + tile) * kStatePanel, smem + kOffD,
                   kStatePanel);
        stores_commit();
        stores_wait_read();
        bar_arrive(kept);
      }
      stores_wait();
    }
  } else if (warp >= 4) {
    // ---- rows ----
    const int quarter = warp % 4, cg = warp / 4 - 1;
    const int row = quarter * 32 + lane, col = col0 + cg * 16, width = p.V - col;
    const bool key = quarter < 2;  // tokens' du; the other half prepares do
    const int t = row & (kDelta - 1);
    const uint32_t mine = (static_cast<uint32_t>(quarter * 32) << 16) + cg * 16;
    float D[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i] = 0.f;
    put_terms(smem + kOffD, kStatePanel, row, cg, D);
    cconv::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(dready);
    const Rows from = key ? p.v : p.d_o;
    const uint16_t* src = from.p + hv * from.sh + col;
    uint4 in[2];
    float4 zin[4];
    auto fetch = [&](int c) {
      const int64_t at = row_a + c * kDelta + t;
      const bool on = c >= 0 && at < row_b;
      load_bf16x16(src + at * from.st, width, on, in);
      if (key) {
        const float4* z = reinterpret_cast<const float4*>(p.z + (at * p.Hv + hv) * p.V + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          zin[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (on && 4 * i < width) zin[i] = z[i];
        }
      }
    };
    fetch(chunks - 1);
    for (int i = 0; i < chunks; ++i) {
      const int st = i % kStages, c = chunks - 1 - i, row0 = row_a + c * kDelta, n = min(kDelta, row_b - row0);
      const float* gates = reinterpret_cast<const float*>(base + st * kStageBytes + kStageKq + kTerms * kJpTerm);
      if (!(ok = DELTA_WARP_WAIT(full + 8 * st, i / kStages))) break;
      const float ef = gates[kEf + t], eb = gates[kEb + t], beta = gates[kBeta + t], total = gates[kTotal];
      if (n < kDelta && t >= n) {
        // rows of the next sequence must not meet K^T and Q^T
        for (int j = cg * 4; j < cg * 4 + 4; ++j)
          for (int k = 0; k < (p.K > kPanelCols ? 2 : 1); ++k)
            sts128(smem + st * kStageBytes + k * kPanelBytes + swizzled(row, j), 0, 0, 0, 0);
      }
      float x[16], y[16];
      unpack16(in, x);  // v, or do
      if (!key) {
        const float f = p.scale * ef;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          sts128(smem + kOffDoRaw + term_piece(t, cg * 2 + j), in[j].x, in[j].y, in[j].z, in[j].w);
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = t < n ? f * x[j] : 0.f;
        put_terms(smem + kOffDo, kTokenPanel, t, cg, y);
        cconv::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(oready);
        fetch(c - 1);
      } else {
        float r[16], z[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[4 * j] = zin[j].x, z[4 * j + 1] = zin[j].y, z[4 * j + 2] = zin[j].z, z[4 * j + 3] = zin[j].w;
        fetch(c - 1);
        if (!(ok = DELTA_WARP_WAIT(acc1, i))) break;
        tc_fence_after();
        load_sum(tmem + mine, r);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          r[j] = t < n ? eb * r[j] : 0.f;
          y[j] = beta * r[j];
        }
        put_terms(smem + kOffDx, kTokenPanel, t, cg, y);
        cconv::fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(xready);
        if (!(ok = DELTA_WARP_WAIT(acc2, i))) break;
        tc_fence_after();
        load_sum(tmem2 + mine, y);
        uint32_t d[16];
        tmem_ld16(tmem2 + 3 * kColumns + mine, d);
        tmem_wait_ld();
        tmem_use16(d);
        float du_z = 0.f, dv_v = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float du = t < n ? r[j] + fmaf(p.scale, __uint_as_float(d[j]), y[j]) : 0.f;
          du_z = fmaf(du, z[j], du_z);
          r[j] = beta * du;
          dv_v = fmaf(r[j], x[j], dv_v);
          y[j] = -ef * r[j];
        }
        put_terms(smem + kOffDx, kTokenPanel, t, cg, y);
        cconv::fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(uready);
        if (t < n) {
          uint16_t* dst = p.dv + (static_cast<int64_t>(row0 + t) * p.Hv + hv) * p.V + col;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = f2_to_bf16x2(f2_pack(r[8 * j + 2 * k], r[8 * j + 2 * k + 1]));
            if (8 * j < width) *reinterpret_cast<uint4*>(dst + 8 * j) = make_uint4(h[0], h[1], h[2], h[3]);
          }
          const int64_t at = (static_cast<int64_t>(tile * 2 + cg) * p.Hv + hv) * p.total + row0 + t;
          p.bdots[at] = du_z;
          p.vdots[at] = dv_v;
        }
      }
      if (i + 1 < chunks || p.dinit) {
        if (!(ok = DELTA_WARP_WAIT(acc3, i))) break;
        tc_fence_after();
        load_sum(tmem + mine, y);
#pragma unroll
        for (int j = 0; j < 16; ++j) D[j] = row < p.K ? fmaf(total, D[j], y[j]) : 0.f;
        if (i + 1 < chunks) {
          if (!(ok = DELTA_WARP_WAIT(kept, i))) break;
          put_terms(smem + kOffD, kStatePanel, row, cg, D);
          cconv::fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(dready);
        }
      }
      if (lane == 0) bar_arrive(empty + 8 * st);
    }
    if (ok && p.dinit && row < p.K) {
      float* dst = p.dinit + ((static_cast<int64_t>(seq) * p.Hv + hv) * p.K + row) * p.V + col;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * i < width)
          *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(D[4 * i], D[4 * i + 1], D[4 * i + 2], D[4 * i + 3]);
    }
  }
  if (!ok) atomicOr(&g_fault_back, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 256);
  }
}

int launch_delta_back(const DeltaCall& c, cudaStream_t stream) {
  BackArgs a{};
  int rc = bind_context();
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc != CCONV_OK) return rc;
  a.v = c.v, a.d_o = c.d_o;
  a.cu = c.cu;
  a.records = c.records;
  a.z = c.z;
  a.ends = c.ends;
  a.vdots = c.vdots, a.bdots = c.bdots;
  a.dv = c.dv, a.dinit = c.dinit;
  a.scale = c.scale;
  a.total = c.s.total, a.nseq = c.s.nseq, a.ratio = c.s.Hv / c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.tiles = delta_tiles(c.s.V);
  const int64_t ctas = static_cast<int64_t>(c.s.nseq) * c.s.Hv * a.tiles;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_delta_back_kernel), kBackBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(cattn_delta_back_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kChainThreads), kBackBytes,
                    stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cattn
