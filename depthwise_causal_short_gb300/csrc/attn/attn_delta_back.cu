// attn_delta_back.cu -- the gated delta rule's chain backwards: the gradient of the state.
//
// The CTAs, rings, terms and roles of attn_delta_chain.cu, from a sequence's last chunk to its first.
// D, the gradient of the state at the chunk's end, is kept as S is there.  A chunk's products:
//   K D                                   -> r' = eb . (K D),  X = beta r'
//   J^T X;  P~^T do                       -> du = r' + J^T X + scale P~^T do,  dv = beta du
//   K^T (-ef . dv);  Q^T (scale ef . do)  -> D = total D + ..
// J and P~ are read from their records with the rows as the contraction, their 64 columns twice over (a
// distance of 0 between the halves of A), so that here too all row warps have results to read.  The
// products that have do in them wait for nothing of the chain; the copying warps prepare do for them.
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
constexpr int kOffD = kRingBytes;
constexpr int kOffDx = kOffD + kTerms * kStatePanel;      // X, then -ef . dv
constexpr int kOffDo = kOffDx + kTerms * kTokenPanel;     // scale ef . do
constexpr int kOffDoRaw = kOffDo + kTerms * kTokenPanel;  // do
constexpr int kOffDots = kOffDoRaw + kTokenPanel;         // [2][4][64] parts of dbeta and v . dv
constexpr int kOffBackBars = kOffDots + 2 * 4 * kDelta * 4;
constexpr int kBackBytes = kOffBackBars + 24 * 8 + 1024;
static_assert(kBackBytes <= 232448, "shared memory of one CTA");

struct BackArgs {
  CUtensorMap mq, mk;
  Rows v, d_o;
  const int32_t* cu;
  const uint8_t* records;
  const float* z;
  uint8_t* ends;          // [slots][Hv][tiles] first terms of D
  float *vdots, *bdots;   // [tiles][Hv][total]
  uint16_t* dv;
  float* dinit;
  float scale;
  int total, nseq, ratio, Hv, K, V, tiles;
};

__global__ void __launch_bounds__(kChainThreads, 1) cattn_delta_back_kernel(const __grid_constant__ BackArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t kqfull = smem + kOffBackBars, recfull = kqfull + 8 * kStages, empty = recfull + 8 * kStages;
  const uint32_t kready = empty + 8 * kStages, oready = kready + 8;                    // by the copying warps
  const uint32_t dready = oready + 8, xready = dready + 8, uready = xready + 8;        // by the rows
  const uint32_t acc1 = uready + 8, acc2 = acc1 + 8, acc3 = acc2 + 8;                  // products
  const uint32_t kept = acc3 + 8, dotsfree = kept + 8, alldone = dotsfree + 8;
  float(*dots)[4][kDelta] = reinterpret_cast<float(*)[4][kDelta]>(base + kOffDots);
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(kqfull + 8 * i, 1);
      bar_init(recfull + 8 * i, 1);
      bar_init(empty + 8 * i, 1 + kRowWarps + kCopyWarps);
    }
    bar_init(kready, kCopyWarps);
    bar_init(oready, kCopyWarps);
    bar_init(dready, kRowWarps);
    bar_init(xready, kRowWarps);
    bar_init(uready, kRowWarps);
    bar_init(acc1, 1);
    bar_init(acc2, 1);
    bar_init(acc3, 1);
    bar_init(kept, 1);
    bar_init(dotsfree, 1);
    bar_init(alldone, 1);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_at, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
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
  const int col0 = tile * kColumns, panels = p.K > kPanelCols ? 2 : 1;
  bool ok = true;

  if (warp == 0) {
    // ---- tiles and records ----
    if (elect_one()) {
      const int hk = hv / p.ratio;
      int i = 0, part = 0;
      for (; i < chunks && ok; ++i) {
        const int st = i % kStages, c = chunks - 1 - i;
        if (i >= kStages && !(ok = DELTA_WAIT(empty + 8 * st, i / kStages - 1))) break;
        if (i > 0 && !(ok = DELTA_WAIT(acc1, i - 1))) break;
        load_kq(smem, kqfull + 8 * st, &p.mk, &p.mq, st, panels, hk, row_a + c * kDelta);
        part = 1;
        if (i > 0 && !(ok = DELTA_WAIT(acc2, i - 1))) break;
        load_record(smem, recfull + 8 * st, p.records + ((slot0 + c) * p.Hv + hv) * kRecordBytes, st);
        part = 0;
      }
      for (int st = 0; st < kStages; ++st) {
        drain(kqfull + 8 * st, (i + part - st + kStages - 1) / kStages);
        drain(recfull + 8 * st, (i - st + kStages - 1) / kStages);
      }
    }
  } else if (warp == 1) {
    // ---- products ----
    if (elect_one()) {
      const int ksteps = (p.K + 15) / 16;
      const uint64_t dd = term_desc(smem + kOffD, kStatePanel), dx = term_desc(smem + kOffDx, kTokenPanel);
      const uint64_t dos = term_desc(smem + kOffDo, kTokenPanel), raw_do = term_desc(smem + kOffDoRaw, kTokenPanel);
      const uint32_t three = mma_desc(3 * kColumns, true, true), two = mma_desc(2 * kColumns, true, true);
      const uint32_t one = mma_desc(kColumns, true, true);
      constexpr uint32_t kThirdX = 2 * kTokenPanel / 16, kTerm = kJpTerm / 16;
      for (int i = 0; i < chunks && ok; ++i) {
        const int st = i % kStages;
        const uint32_t kq = smem + st * kStageKq, rec = smem + kOffRecords + st * kRecordBytes;
        if (!(ok = DELTA_WAIT(kready, i))) break;
        if (!(ok = DELTA_WAIT(dready, i))) break;
        tc_fence_after();
        mma_terms(tmem + kTmAcc1, tmem + kTmK, dd, kStatePanel, ksteps);  // K D
        mma_commit(acc1);
        if (!(ok = DELTA_WAIT(oready, i))) break;
        tc_fence_after();
        const uint64_t dj = tile_desc(rec, 0), dp = tile_desc(rec + kSideBytes, 0);
#pragma unroll 1
        for (int s = 0; s < kTerms; ++s)
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)  // P~^T do
            mma_ss(tmem + kTmOut1, dp + s * kTerm + j * kRowStep, raw_do + j * kTermStep, one, s + j > 0);
        if (!(ok = DELTA_WAIT(xready, i))) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j) {  // J^T X, terms down to 2^-16
          const uint64_t a = dj + j * kRowStep, x = dx + j * kTermStep;
          mma_ss(tmem + kTmAcc2, a, x, two, j > 0);
          mma_ss(tmem + kTmAcc2 + kColumns, a, x + kThirdX, one, true);
          mma_ss(tmem + kTmAcc2, a + kTerm, x, two, true);
          mma_ss(tmem + kTmAcc2 + kColumns, a + 2 * kTerm, x, one, true);
        }
        mma_commit(acc2);
        const bool more = i + 1 < chunks || p.dinit;
        if (more) {
          // (acc1's results were read before xready)
          const uint64_t da = tile_desc(kq + kSideBytes, kPanelBytes);  // Q^T (scale ef . do)
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem + kTmAcc1, da + j * kRowStep, dos + j * kTermStep, three, j > 0);
        }
        if (!(ok = DELTA_WAIT(uready, i))) break;
        tc_fence_after();
        if (more) {
          const uint64_t da = tile_desc(kq, kPanelBytes);  // K^T (-ef . dv)
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem + kTmAcc1, da + j * kRowStep, dx + j * kTermStep, three, true);
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
  } else if (warp == 3) {
    // ---- dbeta and v . dv of the tokens, from their four parts ----
    for (int i = 0; i < chunks; ++i) {
      const int row0 = row_a + (chunks - 1 - i) * kDelta, n = min(kDelta, row_b - row0);
      if (!(ok = DELTA_WARP_WAIT(uready, i))) break;
      float x[2][2];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = j * 32 + lane;
          x[a][j] = (dots[a][0][t] + dots[a][1][t]) + (dots[a][2][t] + dots[a][3][t]);
        }
      __syncwarp();
      if (lane == 0) bar_arrive(dotsfree);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = j * 32 + lane;
        if (t >= n) continue;
        const int64_t at = (static_cast<int64_t>(tile) * p.Hv + hv) * p.total + row0 + t;
        p.bdots[at] = x[0][j];
        p.vdots[at] = x[1][j];
      }
    }
  } else if (warp >= 12) {
    // ---- K to tensor memory; do, raw and scaled, to shared memory ----
    const int quarter = warp % 4, t = (quarter & 1) * 32 + lane, half = quarter >> 1;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int col = col0 + half * 16, width = p.V - col;
    const uint16_t* src = p.d_o.p + hv * p.d_o.sh + col;
    for (int i = 0; i < chunks; ++i) {
      const int st = i % kStages, row0 = row_a + (chunks - 1 - i) * kDelta, n = min(kDelta, row_b - row0);
      uint4 in[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        in[j] = make_uint4(0, 0, 0, 0);
        if (t < n && 8 * j < width)
          in[j] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(row0 + t) * p.d_o.st + 8 * j);
      }
      if (!(ok = DELTA_WARP_WAIT(kqfull + 8 * st, i / kStages))) break;
      if (n < kDelta) {
        // rows of the next sequence must not meet K^T and Q^T
        if (t >= n)
          for (int k = 0; k < panels; ++k)
            for (int j = 0; j < 8; ++j)
              sts128(smem + st * kStageKq + k * kPanelBytes + swizzled(half * kDelta + t, j), 0, 0, 0, 0);
        cconv::fence_proxy_async_smem();
      }
      if (i > 0 && !(ok = DELTA_WARP_WAIT(acc1, i - 1))) break;
      tc_fence_after();
      for (int k = 0; k < panels; ++k)
        copy_row(tmem + lanes + kTmK + 32 * k, smem + st * kStageKq + k * kPanelBytes, t, t < n);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(kready);
      if (!(ok = DELTA_WARP_WAIT(recfull + 8 * st, i / kStages))) break;
      const float f = p.scale * reinterpret_cast<const float*>(base + kOffRecords + st * kRecordBytes + kTerms * kJpTerm)[kEf + t];
      if (i > 0 && !(ok = DELTA_WARP_WAIT(acc3, i - 1))) break;  // the last chunk's do is not needed any more
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x[8];
        sts128(smem + kOffDoRaw + term_piece(t, half * 2 + j), in[j].x, in[j].y, in[j].z, in[j].w);
        unpack8(in[j], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= f;
        put_terms8(smem + kOffDo, kTokenPanel, t, half * 2 + j, x);
      }
      cconv::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(oready);
      if (lane == 0) bar_arrive(empty + 8 * st);
    }
  } else if (warp >= 4) {
    // ---- rows: 16 columns of a channel of D, 8 columns of a token ----
    const int quarter = warp % 4, half = warp / 4 - 1;
    const int row = quarter * 32 + lane, col = col0 + half * 16, width = p.V - col;
    const int t = (quarter & 1) * 32 + lane, piece = (quarter >> 1) * 2 + half;
    const int tcol = col0 + piece * 8;
    const bool there = tcol < p.V;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    float D[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i] = 0.f;
    put_terms(smem + kOffD, kStatePanel, row, half, D);
    cconv::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(dready);
    const uint16_t* v_at = p.v.p + hv * p.v.sh + tcol;
    uint4 vin;
    float4 zin[2];
    auto fetch = [&](int c) {
      const int64_t at = static_cast<int64_t>(row_a) + c * kDelta + t;
      vin = make_uint4(0, 0, 0, 0);
      zin[0] = zin[1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c >= 0 && at < row_b && there) {
        vin = *reinterpret_cast<const uint4*>(v_at + at * p.v.st);
        const float4* z = reinterpret_cast<const float4*>(p.z + (at * p.Hv + hv) * p.V + tcol);
        zin[0] = z[0], zin[1] = z[1];
      }
    };
    fetch(chunks - 1);
    for (int i = 0; i < chunks; ++i) {
      const int st = i % kStages, c = chunks - 1 - i, row0 = row_a + c * kDelta, n = min(kDelta, row_b - row0);
      const float* gates = reinterpret_cast<const float*>(base + kOffRecords + st * kRecordBytes + kTerms * kJpTerm);
      float v[8], r[8], y[8];
      unpack8(vin, v);
      const float z[8] = {zin[0].x, zin[0].y, zin[0].z, zin[0].w, zin[1].x, zin[1].y, zin[1].z, zin[1].w};
      fetch(c - 1);
      if (!(ok = DELTA_WARP_WAIT(recfull + 8 * st, i / kStages))) break;
      const float ef = gates[kEf + t], eb = gates[kEb + t], beta = gates[kBeta + t], total = gates[kTotal];
      if (!(ok = DELTA_WARP_WAIT(acc1, i))) break;
      tc_fence_after();
      load_sum8(tmem + lanes + kTmAcc1 + piece * 8, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = t < n ? eb * r[j] : 0.f;
        y[j] = beta * r[j];
      }
      put_terms8(smem + kOffDx, kTokenPanel, t, piece, y);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(xready);
      if (!(ok = DELTA_WARP_WAIT(acc2, i))) break;
      tc_fence_after();
      uint32_t d[8];
      tmem_ld8(tmem + lanes + kTmOut1 + piece * 8, d);
      load_sum8(tmem + lanes + kTmAcc2 + piece * 8, y);
      tmem_use8(d);
      float du_z = 0.f, dv_v = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float du = t < n ? r[j] + fmaf(p.scale, __uint_as_float(d[j]), y[j]) : 0.f;
        du_z = fmaf(du, z[j], du_z);
        r[j] = beta * du;
        dv_v = fmaf(r[j], v[j], dv_v);
        y[j] = -ef * r[j];
      }
      put_terms8(smem + kOffDx, kTokenPanel, t, piece, y);
      cconv::fence_proxy_async_smem();
      if (i > 0 && !(ok = DELTA_WARP_WAIT(dotsfree, i - 1))) break;
      dots[0][piece][t] = du_z;
      dots[1][piece][t] = dv_v;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(uready);
      if (t < n && there)
        *reinterpret_cast<uint4*>(p.dv + (static_cast<int64_t>(row0 + t) * p.Hv + hv) * p.V + tcol) = pack8(r);
      if (i + 1 < chunks || p.dinit) {
        float x[16];
        if (!(ok = DELTA_WARP_WAIT(acc3, i))) break;
        tc_fence_after();
        load_sum(tmem + lanes + kTmAcc1 + half * 16, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) D[j] = row < p.K ? fmaf(total, D[j], x[j]) : 0.f;
        if (i + 1 < chunks) {
          if (!(ok = DELTA_WARP_WAIT(kept, i))) break;
          put_terms(smem + kOffD, kStatePanel, row, half, D);
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
    tmem_free(tmem, 512);
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
