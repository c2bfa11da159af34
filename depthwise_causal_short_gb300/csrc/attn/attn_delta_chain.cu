// attn_delta_chain.cu -- the gated delta rule's chain over the chunks of a sequence.
//
// A CTA owns 32 columns of V of one sequence and value head (the columns of a state never meet) and
// goes through the chunks; a chunk's record (attn_delta_prep.cu) and its K and Q come through rings of two
// slots.  The state lives in registers in fp32, a row (channel of K) of 16 columns a thread, and as three
// bf16 terms in shared memory.  Three products a chunk, each behind the last:
//   K S            -> r = v - ef . (K S),  X = beta r
//   J X            -> z = r + J X,         u = beta z
//   K^T (eb . u)   -> S = total S + ..
// The three terms of S, X and eb . u lie side by side as columns of one operand, so that A is read once
// for several; the terms' products are added up in registers.  K and J are first operands from tensor
// memory (in shared memory they took 200 cycles a product of 128 x 96 x 16 beside the next chunk's loads),
// copied there by four warps, and in lanes 64 to 127 once more: so all four quarters of the row warps have
// tokens' results to read, 8 columns a thread, where two would have 16.
// What the chain does not wait for, o = scale (ef . (Q S) + P~ X), fills the tensor cores while the rows
// work, and goes out through the copying warps.
// The gradient runs the same chain first (BWD): it leaves z, two terms of u, the first term of every S_0,
// and o . do in place of o.  Its own chain, from the last chunk to the first, is attn_delta_back.cu.
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
constexpr int kOffState = kRingBytes;
constexpr int kOffX = kOffState + kTerms * kStatePanel;
constexpr int kOffU = kOffX + kTerms * kTokenPanel;      // eb . u
constexpr int kOffChainBars = kOffU + kTerms * kTokenPanel;
constexpr int kChainBytes = kOffChainBars + 20 * 8 + 1024;
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
  uint8_t* u;      // [slots][Hv][tiles] two terms of u
  float* dots;     // [tiles][Hv][total] parts of o . do
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
  const uint32_t kqfull = smem + kOffChainBars, recfull = kqfull + 8 * kStages, empty = recfull + 8 * kStages;
  const uint32_t kready = empty + 8 * kStages, jready = kready + 8;                    // operands in tensor memory
  const uint32_t sready = jready + 8, xready = sready + 8, uready = xready + 8;        // and in shared memory
  const uint32_t acc1 = uready + 8, acc2 = acc1 + 8, acc3 = acc2 + 8, outs = acc3 + 8; // products
  const uint32_t outfree = outs + 8, kept = outfree + 8, alldone = kept + 8;
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(kqfull + 8 * i, 1);
      bar_init(recfull + 8 * i, 1);
      bar_init(empty + 8 * i, 1 + kRowWarps + kCopyWarps);
    }
    bar_init(kready, kCopyWarps);
    bar_init(jready, kCopyWarps);
    bar_init(sready, kRowWarps);
    bar_init(xready, kRowWarps);
    bar_init(uready, kRowWarps);
    bar_init(acc1, 1);
    bar_init(acc2, 1);
    bar_init(acc3, 1);
    bar_init(outs, 1);
    bar_init(outfree, kCopyWarps);
    bar_init(kept, 1);
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
  const ChainPlace w = chain_place(p, lane);
  const int chunks = (w.b - w.a + kDelta - 1) / kDelta;
  const bool keep = !BWD && p.fin != nullptr && w.write;  // the state after the last chunk is needed
  const int col0 = w.tile * kColumns;
  const int64_t slot0 = w.a / kDelta + w.seq;
  const int panels = p.K > kPanelCols ? 2 : 1;
  bool ok = true;

  if (warp == 0) {
    // ---- tiles and records: the next chunk's while this one's products wait for the rows ----
    if (elect_one()) {
      const int hk = w.hv / p.ratio;
      int c = 0, part = 0;
      for (; c < chunks && ok; ++c) {
        const int st = c % kStages;
        if (c >= kStages && !(ok = DELTA_WAIT(empty + 8 * st, c / kStages - 1))) break;
        if (c > 0 && !(ok = DELTA_WAIT(acc1, c - 1))) break;
        load_kq(smem, kqfull + 8 * st, &p.mk, &p.mq, st, panels, hk, w.a + c * kDelta);
        part = 1;
        if (c > 0 && !(ok = DELTA_WAIT(acc2, c - 1))) break;
        load_record(smem, recfull + 8 * st, p.records + ((slot0 + c) * p.Hv + w.hv) * kRecordBytes, st);
        part = 0;
      }
      for (int st = 0; st < kStages; ++st) {
        drain(kqfull + 8 * st, (c + part - st + kStages - 1) / kStages);
        drain(recfull + 8 * st, (c - st + kStages - 1) / kStages);
      }
    }
  } else if (warp == 1) {
    // ---- products ----
    if (elect_one()) {
      const int ksteps = (p.K + 15) / 16;
      const uint64_t ds = term_desc(smem + kOffState, kStatePanel), dx = term_desc(smem + kOffX, kTokenPanel);
      const uint64_t du = term_desc(smem + kOffU, kTokenPanel);
      const uint32_t two = mma_desc(2 * kColumns, false, true), one = mma_desc(kColumns, false, true);
      constexpr uint32_t kThirdS = 2 * kStatePanel / 16, kThirdX = 2 * kTokenPanel / 16;
      for (int c = 0; c < chunks && ok; ++c) {
        const int st = c % kStages;
        const uint32_t kq = smem + st * kStageKq, rec = smem + kOffRecords + st * kRecordBytes;
        if (!(ok = DELTA_WAIT(kready, c))) break;
        if (!(ok = DELTA_WAIT(sready, c))) break;
        tc_fence_after();
        mma_terms(tmem + kTmAcc1, tmem + kTmK, ds, kStatePanel, ksteps);  // K S
        mma_commit(acc1);
        if (c > 0 && !(ok = DELTA_WAIT(outfree, c - 1))) break;
        tc_fence_after();
        // Q S (lanes 64 to 127 of this and of P~ X, made of what follows in shared memory, are not read)
        const uint64_t dq = tile_desc(kq + kSideBytes, 0);
#pragma unroll 1
        for (int j = 0; j < ksteps; ++j) {
          mma_ss(tmem + kTmOut1, dq + col_step(j), ds + j * kTermStep, two, j > 0);
          if (BWD) mma_ss(tmem + kTmOut1 + kColumns, dq + col_step(j), ds + kThirdS + j * kTermStep, one, true);
        }
        if (!(ok = DELTA_WAIT(jready, c))) break;
        if (!(ok = DELTA_WAIT(xready, c))) break;
        tc_fence_after();
        // J X, terms down to 2^-16
        mma_terms(tmem + kTmAcc2, tmem + kTmJ, dx, kTokenPanel, kDelta / 16);
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j) {
          mma_ts(tmem + kTmAcc2, tmem + kTmJ + 32 + j * 8, dx + j * kTermStep, two, true);
          mma_ts(tmem + kTmAcc2 + kColumns, tmem + kTmJ + 64 + j * 8, dx + j * kTermStep, one, true);
        }
        mma_commit(acc2);
        // P~ X: with two terms o is as exact as its store; o . do takes all
        const uint64_t dp = tile_desc(rec + kSideBytes, 0);
        constexpr uint32_t kTerm = kJpTerm / 16;
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j) {
          const uint64_t x = dx + j * kTermStep;
          mma_ss(tmem + kTmOut2, dp + 2 * j, x, two, j > 0);
          mma_ss(tmem + kTmOut2, dp + kTerm + 2 * j, x, BWD ? two : one, true);
          if (BWD) {
            mma_ss(tmem + kTmOut2 + kColumns, dp + 2 * j, x + kThirdX, one, true);
            mma_ss(tmem + kTmOut2 + kColumns, dp + 2 * kTerm + 2 * j, x, one, true);
          }
        }
        mma_commit(outs);
        if (!(ok = DELTA_WAIT(uready, c))) break;
        tc_fence_after();
        if (c + 1 < chunks || keep) {
          const uint64_t da = tile_desc(kq, kPanelBytes);  // K^T (eb . u)
          const uint32_t desc = mma_desc(3 * kColumns, true, true);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem + kTmAcc1, da + j * kRowStep, du + j * kTermStep, desc, j > 0);
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
  } else if (warp >= 12) {
    // ---- copies to tensor memory, and the outputs ----
    const int quarter = warp % 4, t = (quarter & 1) * 32 + lane;  // K and J twice, in lanes 0 and 64 on
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const Rows from = p.d_o;
    const int width = p.V - col0;
    for (int c = -1; c < chunks; ++c) {
      const int next = c + 1, st = next % kStages;
      if (next < chunks) {
        const int n = min(kDelta, w.b - w.a - next * kDelta);
        if (!(ok = DELTA_WARP_WAIT(kqfull + 8 * st, next / kStages))) break;
        if (n < kDelta && t >= n && quarter < 2) {
          // rows of the next sequence must not meet K^T (eb . u), where 0 * NaN is not 0
          for (int k = 0; k < panels; ++k)
            for (int i = 0; i < 8; ++i) sts128(smem + st * kStageKq + k * kPanelBytes + swizzled(t, i), 0, 0, 0, 0);
        }
        if (n < kDelta) cconv::fence_proxy_async_smem();
        if (c >= 0 && !(ok = DELTA_WARP_WAIT(acc1, c))) break;
        tc_fence_after();
        for (int k = 0; k < panels; ++k)
          copy_row(tmem + lanes + kTmK + 32 * k, smem + st * kStageKq + k * kPanelBytes, t, t < n);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(kready);
      }
      if (c >= 0) {
      const int row0 = w.a + c * kDelta, here = c % kStages;
      const bool on = quarter < 2 && row0 + t < w.b;
      uint4 in[4];
      if (BWD)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          in[i] = make_uint4(0, 0, 0, 0);
          if (on && 8 * i < width)
            in[i] = *reinterpret_cast<const uint4*>(from.p + static_cast<int64_t>(row0 + t) * from.st + w.hv * from.sh +
                                                    col0 + 8 * i);
        }
      const float ef = reinterpret_cast<const float*>(base + kOffRecords + here * kRecordBytes + kTerms * kJpTerm)[kEf + t];
      if (!(ok = DELTA_WARP_WAIT(outs, c))) break;
      tc_fence_after();
      float sum = 0.f;
      if (quarter < 2) {
        uint16_t* dst = p.o + (static_cast<int64_t>(row0 + t) * p.Hv + w.hv) * p.V + col0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a[8], b[8];
          load_sum8(tmem + lanes + kTmOut1 + 8 * i, a);
          load_sum8(tmem + lanes + kTmOut2 + 8 * i, b);
          float d[8];
          if (BWD) unpack8(in[i], d);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            a[j] = p.scale * fmaf(ef, a[j], b[j]);
            if (BWD) sum = fmaf(a[j], d[j], sum);
          }
          if (!BWD && on && 8 * i < width) *reinterpret_cast<uint4*>(dst + 8 * i) = pack8(a);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(outfree);
      if (lane == 0) bar_arrive(empty + 8 * here);
      if (BWD && on) p.dots[(static_cast<int64_t>(w.tile) * p.Hv + w.hv) * p.total + row0 + t] = sum;
      }
      if (next < chunks) {
        if (!(ok = DELTA_WARP_WAIT(recfull + 8 * st, next / kStages))) break;
        if (c >= 0 && !(ok = DELTA_WARP_WAIT(acc2, c))) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < kTerms; ++i)
          copy_row(tmem + lanes + kTmJ + 32 * i, smem + kOffRecords + st * kRecordBytes + i * kJpTerm, t, true);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(jready);
      }
    }
  } else if (warp >= 4) {
    // ---- rows: 16 columns of a channel's state, 8 columns of a token ----
    const int quarter = warp % 4, half = warp / 4 - 1;   // lanes of TMEM, column group
    const int row = quarter * 32 + lane, col = col0 + half * 16, width = p.V - col;
    const int t = (quarter & 1) * 32 + lane, piece = (quarter >> 1) * 2 + half;
    const int tcol = col0 + piece * 8;
    const bool there = tcol < p.V;                       // the token's columns
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
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
    put_terms(smem + kOffState, kStatePanel, row, half, S);
    cconv::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(sready);
    const uint16_t* v_at = p.v.p + w.hv * p.v.sh + tcol;
    auto fetch = [&](int c) {
      const int64_t at = static_cast<int64_t>(w.a) + c * kDelta + t;
      return there && at < w.b ? *reinterpret_cast<const uint4*>(v_at + at * p.v.st) : make_uint4(0, 0, 0, 0);
    };
    uint4 next = fetch(0);
    for (int c = 0; c < chunks; ++c) {
      const int st = c % kStages, row0 = w.a + c * kDelta, n = min(kDelta, w.b - row0);
      const float* gates = reinterpret_cast<const float*>(base + kOffRecords + st * kRecordBytes + kTerms * kJpTerm);
      float r[8], y[8];
      unpack8(next, r);
      next = fetch(c + 1);
      if (!(ok = DELTA_WARP_WAIT(recfull + 8 * st, c / kStages))) break;
      const float ef = gates[kEf + t], eb = gates[kEb + t], beta = gates[kBeta + t], total = gates[kTotal];
      if (!(ok = DELTA_WARP_WAIT(acc1, c))) break;
      tc_fence_after();
      load_sum8(tmem + lanes + kTmAcc1 + piece * 8, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = t < n ? fmaf(-ef, y[i], r[i]) : 0.f;
        y[i] = beta * r[i];
      }
      put_terms8(smem + kOffX, kTokenPanel, t, piece, y);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(xready);
      if (!(ok = DELTA_WARP_WAIT(acc2, c))) break;
      tc_fence_after();
      load_sum8(tmem + lanes + kTmAcc2 + piece * 8, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] += y[i];
        y[i] = t < n ? eb * (beta * r[i]) : 0.f;
      }
      put_terms8(smem + kOffU, kTokenPanel, t, piece, y);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(uready);
      if (BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = t < n ? beta * r[i] : 0.f;
        uint4 u[kTerms];
        split8(y, u);
        uint8_t* tile = p.u + (((slot0 + c) * p.Hv + w.hv) * p.tiles + w.tile) * kUTile + term_piece(t, piece);
        *reinterpret_cast<uint4*>(tile) = u[0];
        *reinterpret_cast<uint4*>(tile + kTokenPanel) = u[1];
        if (t < n && there) {
          float4* dst = reinterpret_cast<float4*>(p.z + (static_cast<int64_t>(row0 + t) * p.Hv + w.hv) * p.V + tcol);
          dst[0] = make_float4(r[0], r[1], r[2], r[3]);
          dst[1] = make_float4(r[4], r[5], r[6], r[7]);
        }
      }
      if (c + 1 < chunks || keep) {
        float x[16];
        if (!(ok = DELTA_WARP_WAIT(acc3, c))) break;
        tc_fence_after();
        load_sum(tmem + lanes + kTmAcc1 + half * 16, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = row < p.K ? fmaf(total, S[i], x[i]) : 0.f;
        if (c + 1 < chunks) {
          if (BWD && !(ok = DELTA_WARP_WAIT(kept, c))) break;
          put_terms(smem + kOffState, kStatePanel, row, half, S);
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
    tmem_free(tmem, 512);
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
  a.z = c.z, a.u = c.u, a.heads = c.heads, a.dots = c.odots;
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
