// attn_delta_chain.cu -- the gated delta rule's chain over the chunks of a sequence.
//
// A CTA owns 32 columns of V of one sequence and value head (the columns of a state never meet) and
// goes through the chunks; the chunk's record (attn_delta_prep.cu) comes through a ring of two slots
// together with its K and Q.  The state lives in registers in fp32, a row (channel of K) of 16 columns
// a thread, and as three bf16 terms in shared memory.  Three products a chunk, each behind the last:
//   [K; Q] S          -> r = v - ef . (K S),  X = beta r;   ef . (Q S)
//   [J; P~] X         -> z = r + J X,  u = beta z;          o = scale (ef . (Q S) + P~ X)
//   K^T (eb . u)      -> S = total S + ..
// The gradient runs the same chain first (BWD): it leaves z, the first term of every S_0 and o . do in
// place of o.  Its own chain, from the last chunk to the first, is attn_delta_back.cu.
//
// The three terms of S, X and eb . u lie side by side as columns of one operand (N = 96), and their
// products are added up in registers: A is read once for all three.
//
// Bound by that chain: a product, its results to registers, the next operand to shared memory.
#include <cudaTypedefs.h>

#include "attn_chunk_host.h"
#include "attn_delta.cuh"

namespace cattn {

static __device__ unsigned g_fault_chain;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_chain, sizeof(*out))) != cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_chain, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

// shared memory, from a 1024-byte boundary
constexpr int kOffState = kStages * kStageBytes;
constexpr int kOffX = kOffState + kTerms * kStatePanel;  // X, then eb . u
constexpr int kOffChainBars = kOffX + kTerms * kTokenPanel;
constexpr int kChainBytes = kOffChainBars + 16 * 8 + 1024;
static_assert(kChainBytes <= 232448, "shared memory of one CTA");

struct ChainArgs {
  CUtensorMap mq, mk;
  Rows v, d_o;
  const int32_t* cu;
  Slots slots;
  int32_t* status;
  const float* initial;
  float* fin;
  uint16_t* o;
  const uint8_t* records;
  float* z;        // [total][Hv][V]
  uint8_t* heads;  // [slots][Hv][tiles] first terms of S_0
  float* dots;     // [2 tiles][Hv][total] parts of o . do
  float scale;
  int total, nseq, ratio, Hv, K, V, tiles, checked;
};

// This CTA's sequence: its rows, and the state slot (-1: none that can be used).
struct ChainPlace {
  int seq, hv, tile, a, b;
  int64_t slot;
  bool write;  // the state indices are valid
};
__device__ __forceinline__ ChainPlace chain_place(const ChainArgs& p, int lane) {
  ChainPlace w;
  w.tile = static_cast<int>(blockIdx.x % p.tiles);
  w.hv = static_cast<int>(blockIdx.x / p.tiles % p.Hv);
  w.seq = static_cast<int>(blockIdx.x / p.tiles / p.Hv);
  const int a = p.cu[w.seq], b = p.cu[w.seq + 1];
  sequence_rows(p.cu, w.seq, p.total, w.a, w.b);
  const bool bad = b < a || (w.seq == 0 && a != 0) || (w.seq == p.nseq - 1 && b != p.total) || a < 0 || b > p.total;
  if (bad) {
    w.b = w.a;
    if (threadIdx.x == 0) atomicOr(&g_fault_chain, kFaultSeqlens);
  }
  w.slot = p.slots.of(w.seq);
  w.write = true;
  if (p.slots.idx) {
    if (p.checked) {
      w.write = p.status[0] == CCONV_OK;
    } else {
      const unsigned off = check_indices(lane < p.nseq ? p.slots.idx[lane] : -1, p.nseq, p.slots.S, false, lane);
      w.write = off == 0;
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.status[0] = off ? CCONV_ERR_INDEX : CCONV_OK;
        p.status[1] = static_cast<int>(off);
      }
    }
  }
  return w;
}

template <bool BWD>
__global__ void __launch_bounds__(kChainThreads, 1) cattn_delta_chain_kernel(const __grid_constant__ ChainArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t full = smem + kOffChainBars, empty = full + 8 * kStages;
  const uint32_t sready = empty + 8 * kStages, xready = sready + 8, uready = xready + 8;
  const uint32_t acc1 = uready + 8, acc2 = acc1 + 8, acc3 = acc2 + 8, alldone = acc3 + 8;
  const uint32_t kept = alldone + 8;
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1 + kRowWarps);
    }
    bar_init(sready, kRowWarps);
    bar_init(xready, kRowWarps);
    bar_init(uready, kRowWarps);
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
  const ChainPlace w = chain_place(p, lane);
  const int chunks = (w.b - w.a + kDelta - 1) / kDelta;
  const bool keep = !BWD && p.fin != nullptr && w.write;  // the state after the last chunk is needed
  const int col0 = w.tile * kColumns;
  bool ok = true;

  if (warp == 0) {
    // ---- tiles and records ----
    if (elect_one()) {
      const int panels = p.K > kPanelCols ? 2 : 1, hk = w.hv / p.ratio;
      const int64_t slot0 = w.a / kDelta + w.seq;
      int c = 0;
      for (; c < chunks && ok; ++c) {
        const int st = c % kStages;
        if (c >= kStages && !(ok = DELTA_WAIT(empty + 8 * st, c / kStages - 1))) break;
        const uint32_t at = smem + st * kStageBytes, bar = full + 8 * st;
        bar_expect(bar, panels * 2 * kSideBytes + kRecordBytes);
#pragma unroll 1
        for (int i = 0; i < panels; ++i) {
          load_box(at + i * kPanelBytes, &p.mk, bar, i * kPanelCols, hk, w.a + c * kDelta);
          load_box(at + i * kPanelBytes + kSideBytes, &p.mq, bar, i * kPanelCols, hk, w.a + c * kDelta);
        }
        bulk_load(at + kStageKq, p.records + ((slot0 + c) * p.Hv + w.hv) * kRecordBytes, kRecordBytes, bar);
      }
      for (int st = 0; st < kStages; ++st) drain(full + 8 * st, (c - st + kStages - 1) / kStages);
    }
  } else if (warp == 1) {
    // ---- products ----
    if (elect_one()) {
      const int ksteps = (p.K + 15) / 16;
      const uint64_t ds = term_desc(smem + kOffState, kStatePanel), dx = term_desc(smem + kOffX, kTokenPanel);
      const uint32_t wide = mma_desc(3 * kColumns, false, true);
      for (int c = 0; c < chunks && ok; ++c) {
        const int st = c % kStages;
        const uint32_t at = smem + st * kStageBytes;
        if (!(ok = DELTA_WAIT(full + 8 * st, c / kStages))) break;
        if (!(ok = DELTA_WAIT(sready, c))) break;
        tc_fence_after();
        const uint64_t dkq = tile_desc(at, 0);
#pragma unroll 1
        for (int j = 0; j < ksteps; ++j) mma_ss(tmem, dkq + col_step(j), ds + j * kTermStep, wide, j > 0);
        mma_commit(acc1);
        if (!(ok = DELTA_WAIT(xready, c))) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < kTerms; ++i) {
          const uint64_t da = tile_desc(at + kStageKq + i * kJpTerm, 0);
          const uint32_t desc = mma_desc((kTerms - i) * kColumns, false, true);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem2, da + 2 * j, dx + j * kTermStep, desc, i + j > 0);
        }
        mma_commit(acc2);
        if (!(ok = DELTA_WAIT(uready, c))) break;
        tc_fence_after();
        if (c + 1 < chunks || keep) {
          const uint64_t da = tile_desc(at, kPanelBytes);
          const uint32_t desc = mma_desc(3 * kColumns, true, true);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j) mma_ss(tmem, da + j * kRowStep, dx + j * kTermStep, desc, j > 0);
          mma_commit(acc3);
        }
        mma_commit(empty + 8 * st);
      }
      // nothing of this CTA may be in flight when its shared memory and TMEM go
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (BWD && warp == 2) {
    // ---- the first term of every S_0 ----
    if (elect_one()) {
      const int64_t slot0 = w.a / kDelta + w.seq;
      for (int c = 0; c < chunks && ok; ++c) {
        if (!(ok = DELTA_WAIT(sready, c))) break;
        bulk_store(p.heads + (((slot0 + c) * p.Hv + w.hv) * p.tiles + w.tile) * kStatePanel, smem + kOffState,
                   kStatePanel);
        stores_commit();
        stores_wait_read();
        bar_arrive(kept);
      }
      stores_wait();
    }
  } else if (warp >= 4) {
    // ---- rows ----
    const int quarter = warp % 4, cg = warp / 4 - 1;     // lanes of TMEM, column group
    const int row = quarter * 32 + lane, col = col0 + cg * 16;
    const int width = p.V - col;                          // columns of this thread that there are
    const bool key = quarter < 2;                         // row of K (token) or of Q
    const int t = row & (kDelta - 1);
    const uint32_t mine = (static_cast<uint32_t>(quarter * 32) << 16) + cg * 16;
    float S[16];
    {
      const bool has = p.initial && w.slot >= 0 && row < p.K;
      const float* src = p.initial + ((w.slot * p.Hv + w.hv) * p.K + row) * p.V + col;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (has && 4 * i < width) x = *reinterpret_cast<const float4*>(src + 4 * i);
        S[4 * i] = x.x, S[4 * i + 1] = x.y, S[4 * i + 2] = x.z, S[4 * i + 3] = x.w;
      }
    }
    put_terms(smem + kOffState, kStatePanel, row, cg, S);
    cconv::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(sready);
    const Rows from = key ? p.v : p.d_o;  // rows of v, or (BWD) of do
    const uint16_t* v_at = from.p + w.hv * from.sh + col;
    uint4 vraw[2];
    if (key || BWD) load_bf16x16(v_at + static_cast<int64_t>(w.a + t) * from.st, width, t < w.b - w.a, vraw);
    for (int c = 0; c < chunks; ++c) {
      const int st = c % kStages, row0 = w.a + c * kDelta, n = min(kDelta, w.b - row0);
      const float* gates = reinterpret_cast<const float*>(base + st * kStageBytes + kStageKq + kTerms * kJpTerm);
      if (!(ok = DELTA_WARP_WAIT(full + 8 * st, c / kStages))) break;
      const float ef = gates[kEf + t], eb = gates[kEb + t], beta = gates[kBeta + t], total = gates[kTotal];
      float r[16], y[16];
      if (!(ok = DELTA_WARP_WAIT(acc1, c))) break;
      tc_fence_after();
      load_sum(tmem + mine, y);
      if (key) {
        float x[16];
        unpack16(vraw, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          r[i] = t < n ? fmaf(-ef, y[i], r[i]) : 0.f;
          x[i] = beta * r[i];
        }
        put_terms(smem + kOffX, kTokenPanel, t, cg, x);
        if (n < kDelta && t >= n) {
          // rows of the next sequence must not meet K^T (eb . u), where 0 * NaN is not 0
          for (int i = cg * 4; i < cg * 4 + 4; ++i)
            for (int k = 0; k < (p.K > kPanelCols ? 2 : 1); ++k)
              sts128(smem + st * kStageBytes + k * kPanelBytes + swizzled(t, i), 0, 0, 0, 0);
        }
        cconv::fence_proxy_async_smem();
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = ef * y[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(xready);
      uint4 doraw[2] = {vraw[0], vraw[1]};
      if ((key || BWD) && c + 1 < chunks)
        load_bf16x16(v_at + static_cast<int64_t>(row0 + kDelta + t) * from.st, width, row0 + kDelta + t < w.b, vraw);
      if (!(ok = DELTA_WARP_WAIT(acc2, c))) break;
      tc_fence_after();
      load_sum(tmem2 + mine, y);
      if (key) {
        const float f = eb * beta;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          r[i] += y[i];
          y[i] = t < n ? f * r[i] : 0.f;
        }
        put_terms(smem + kOffX, kTokenPanel, t, cg, y);
        cconv::fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(uready);
      if (BWD && t < n) {
        if (key) {
          float* dst = p.z + (static_cast<int64_t>(row0 + t) * p.Hv + w.hv) * p.V + col;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * i < width)
              *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
        } else {
          float d[16], sum = 0.f;
          unpack16(doraw, d);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum = fmaf(d[i], r[i] + y[i], sum);
          p.dots[(static_cast<int64_t>(w.tile * 2 + cg) * p.Hv + w.hv) * p.total + row0 + t] = p.scale * sum;
        }
      }
      if (!BWD && !key && t < n) {
        uint16_t* dst = p.o + (static_cast<int64_t>(row0 + t) * p.Hv + w.hv) * p.V + col;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t h[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[j] = f2_to_bf16x2(f2_pack(p.scale * (r[8 * i + 2 * j] + y[8 * i + 2 * j]),
                                        p.scale * (r[8 * i + 2 * j + 1] + y[8 * i + 2 * j + 1])));
          if (8 * i < width) *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      if (c + 1 < chunks || keep) {
        if (!(ok = DELTA_WARP_WAIT(acc3, c))) break;
        tc_fence_after();
        load_sum(tmem + mine, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = row < p.K ? fmaf(total, S[i], y[i]) : 0.f;
        if (c + 1 < chunks) {
          if (BWD && !(ok = DELTA_WARP_WAIT(kept, c))) break;
          put_terms(smem + kOffState, kStatePanel, row, cg, S);
          cconv::fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(sready);
        }
      }
      if (lane == 0) bar_arrive(empty + 8 * st);
    }
    if (ok && keep && w.slot >= 0 && row < p.K) {
      float* dst = p.fin + ((w.slot * p.Hv + w.hv) * p.K + row) * p.V + col;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * i < width) *reinterpret_cast<float4*>(dst + 4 * i) = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
    }
  }
  if (!ok) atomicOr(&g_fault_chain, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 256);
  }
}

template <bool BWD>
static int launch_chain(const DeltaCall& c, cudaStream_t stream) {
  ChainArgs a{};
  int rc = CCONV_OK;
  if (c.s.total > 0) {
    rc = bind_context();
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, kDelta);
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, kDelta);
    if (rc != CCONV_OK) return rc;
  }
  a.v = c.v, a.d_o = c.d_o;
  a.cu = c.cu, a.slots = c.slots, a.status = c.status, a.checked = c.checked;
  a.initial = c.initial, a.fin = c.fin;
  a.o = c.o;
  a.records = c.records;
  a.z = c.z, a.heads = c.heads, a.dots = c.odots;
  a.scale = c.scale;
  a.total = c.s.total, a.nseq = c.s.nseq, a.ratio = c.s.Hv / c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.tiles = delta_tiles(c.s.V);
  auto kern = cattn_delta_chain_kernel<BWD>;
  const int64_t ctas = static_cast<int64_t>(c.s.nseq) * c.s.Hv * a.tiles;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kChainBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kChainThreads), kChainBytes, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_delta_fwd(const DeltaCall& c, cudaStream_t stream) { return launch_chain<false>(c, stream); }
int launch_delta_states(const DeltaCall& c, cudaStream_t stream) { return launch_chain<true>(c, stream); }

}  // namespace cattn
