// attn_delta_chain.cuh -- the gated delta rule's chain over the chunks of a sequence.
//
// A CTA owns 32 columns of V of one sequence and value head (the columns of a state never meet) and
// goes through the chunks; a chunk's K and Q and its record (attn_delta_prep.cu) come through a ring of two
// slots.  The state lives in registers in fp32, a row (channel of K) of 16 columns a thread, and as three
// bf16 terms in shared memory.  Three products a chunk, each behind the last:
//   [K; Q] S       -> r = v - ef . (K S),  X = beta r;   ef . (Q S)
//   [J; P~] X      -> z = r + J X,  u = beta z;          o = scale (ef . (Q S) + P~ X)
//   K^T (eb . u)   -> S = total S + ..
// The three terms of S, X and eb . u lie side by side as columns of one operand (N = 96), so that A is
// read once for all three; their products are added up in registers.
// The gradient runs the same chain first (BWD): it leaves z, two terms of u and of every S_0 (and
// every kAnchorChunks-th in fp32), and o . do in place of o.  Its own chain, from the last chunk to the first,
// is attn_delta_back.cuh.
//
// Bound by that chain: a product, its results to registers, the next operand to shared memory.  2 sequences of
// 8192 rows, 16 heads of 128 x 128 (128 CTAs, 128 chunks each): 290 us, 360 BWD; 4200 to 4600 cycles a chunk, of which
// the three products take 1600 and their operands some 1400 between them.  Tensor cores are busy 15 to 18 % of the
// time, memory 17 to 33 %.  A CTA is one on its
// SM (204 KB); 28 warps in place of 12 were slower, and so was A from shared memory (by a tenth).
#pragma once

#include <cudaTypedefs.h>

#include "attn_chunk_host.h"
#include "attn_delta.cuh"

namespace cattn {
namespace chain {

constexpr int kThreads = (4 + kRowWarps) * 32;
// shared memory, from a 1024-byte boundary: a ring of two slots
constexpr int kOffState = 2 * kSlotBytes;
constexpr int kOffX = kOffState + kTerms * kStatePanel;  // X, then eb . u
constexpr int kOffBars = kOffX + kTerms * kTokenPanel;
constexpr int kBytes = kOffBars + 24 * 8 + 1024;
static_assert(kBytes <= 232448, "shared memory of one CTA");
// columns of tensor memory: three accumulators of three terms, [K; Q], [J; P~]
constexpr int kTmFirst = 0, kTmSecond = 96, kTmThird = 192, kTmKq = 288, kTmJp = 352;

struct Args {
  CUtensorMap mq, mk;
  Rows v, d_o;
  const int32_t* cu;
  Slots slots;
  int32_t* status;
  const float* initial;
  float* fin;
  uint16_t* o;
  const uint8_t* records;
  float* z;        // [slots][Hv][tiles], see pairs_at
  uint8_t* heads;  // [slots][Hv][tiles] two terms of S_0
  uint8_t* u;      // [slots][Hv][tiles] two terms of u
  float* dots;     // [2 tiles][Hv][total] parts of o . do
  float* anchors;  // [anchors][Hv][tiles] of kAnchorFloats: S_0 of every kAnchorChunks-th chunk
  float scale;
  int total, nseq, ratio, Hv, K, V, tiles, checked;
};

// This CTA's sequence: its rows, and the state slot (-1: none that can be used).
struct Place {
  int seq, hv, tile, a, b;
  int64_t slot;
  bool write;  // the state indices are valid
};
__device__ __forceinline__ Place place_of(const Args& p, int cta, int lane, unsigned* fault) {
  Place w;
  w.tile = cta % p.tiles;
  w.hv = cta / p.tiles % p.Hv;
  w.seq = cta / p.tiles / p.Hv;
  const int a = p.cu[w.seq], b = p.cu[w.seq + 1];
  sequence_rows(p.cu, w.seq, p.total, w.a, w.b);
  const bool bad = b < a || (w.seq == 0 && a != 0) || (w.seq == p.nseq - 1 && b != p.total) || a < 0 || b > p.total;
  if (bad) {
    w.b = w.a;
    if (threadIdx.x == 0) atomicOr(fault, kFaultSeqlens);
  }
  w.slot = p.slots.of(w.seq);
  w.write = true;
  if (p.slots.idx) {
    if (p.checked) {
      w.write = p.status[0] == CCONV_OK;
    } else {
      const unsigned off = check_indices(lane < p.nseq ? p.slots.idx[lane] : -1, p.nseq, p.slots.S, false, lane);
      w.write = off == 0;
      if (cta == 0 && threadIdx.x == 0) {
        p.status[0] = off ? CCONV_ERR_INDEX : CCONV_OK;
        p.status[1] = static_cast<int>(off);
      }
    }
  }
  return w;
}

// CTA `cta` of the chain, all threads of it (those beyond kThreads have no part).
template <bool BWD>
__device__ __forceinline__ void run(const Args& p, int cta, unsigned* fault) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t kfull = smem + kOffBars, rfull = kfull + 16, empty = rfull + 16;
  const uint32_t sready = empty + 16, xready = sready + 8, uready = xready + 8;
  const uint32_t acc1 = uready + 8, acc2 = acc1 + 8, acc3 = acc2 + 8;
  const uint32_t kept = acc3 + 8, alldone = kept + 8;
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(kfull + 8 * i, 1);
      bar_init(rfull + 8 * i, 1);
      bar_init(empty + 8 * i, 1 + kRowWarps);
    }
    bar_init(sready, kRowWarps);
    bar_init(xready, kRowWarps);
    bar_init(uready, kRowWarps);
    bar_init(acc1, 1);
    bar_init(acc2, 1);
    bar_init(acc3, 1);
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
  const Place w = place_of(p, cta, lane, fault);
  const int chunks = (w.b - w.a + kDelta - 1) / kDelta;
  const bool keep = !BWD && p.fin != nullptr && w.write;  // the state after the last chunk is needed
  const int col0 = w.tile * kColumns;
  const int64_t slot0 = w.a / kDelta + w.seq;
  const int panels = p.K > kPanelCols ? 2 : 1;
  bool ok = true;

  if (warp == 0) {
    // ---- K, Q and records: the next chunk's, each while this one's products wait for the rows (beside
    // a product, they and its reads of shared memory held each other up) ----
    if (elect_one()) {
      const int hk = w.hv / p.ratio;
      int c = 0, part = 0;
      for (; c < chunks && ok; ++c) {
        const int st = c & 1;
        const uint32_t slot = smem + st * kSlotBytes;
        if (c >= 2 && !(ok = DELTA_WAIT(empty + 8 * st, c / 2 - 1))) break;
        if (c > 0 && !(ok = DELTA_WAIT(acc1, c - 1))) break;
        load_kq(slot, kfull + 8 * st, &p.mk, &p.mq, panels, hk, w.a + c * kDelta);
        part = 1;
        if (c > 0 && !(ok = DELTA_WAIT(acc2, c - 1))) break;
        bar_expect(rfull + 8 * st, kRecordBytes);
        bulk_load(slot + kSlotKq, p.records + ((slot0 + c) * p.Hv + w.hv) * kRecordBytes, kRecordBytes, rfull + 8 * st);
        part = 0;
      }
      for (int st = 0; st < 2; ++st) {
        drain(kfull + 8 * st, (c + part - st + 1) / 2);
        drain(rfull + 8 * st, (c - st + 1) / 2);
      }
    }
  } else if (warp == 1) {
    // ---- products ----
    if (elect_one()) {
      const int ksteps = (p.K + 15) / 16;
      const uint64_t ds = term_desc(smem + kOffState, kStatePanel), dx = term_desc(smem + kOffX, kTokenPanel);
      const uint32_t all = mma_desc(kTerms * kColumns, false, true), less = mma_desc((kTerms - 1) * kColumns, false, true);
      const uint32_t one = mma_desc(kColumns, false, true);
      const uint32_t last = mma_desc(kTerms * kColumns, true, true);
      auto copy_kq = [&](int c) {
        const int st = c & 1;
        if (!(ok = DELTA_WAIT(kfull + 8 * st, c / 2))) return;
        const uint64_t dkq = tile_desc(smem + st * kSlotBytes, 0);
#pragma unroll 1
        for (int j = 0; j < ksteps; ++j) tmem_copy(tmem + kTmKq + 8 * j, dkq + col_step(j));
      };
      if (chunks > 0) copy_kq(0);
      for (int c = 0; c < chunks && ok; ++c) {
        const int st = c & 1;
        const uint32_t slot = smem + st * kSlotBytes;
        if (!(ok = DELTA_WAIT(sready, c))) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < ksteps; ++j)  // [K; Q] S
          mma_ts(tmem + kTmFirst, tmem + kTmKq + 8 * j, ds + j * kTermStep, all, j > 0);
        mma_commit(acc1);
        if (!(ok = DELTA_WAIT(rfull + 8 * st, c / 2))) break;
        const uint64_t djp = record_desc(slot + kSlotKq, false);
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j) {
          tmem_copy(tmem + kTmJp + 8 * j, djp + j * kRecordCols);
          tmem_copy(tmem + kTmJp + 32 + 8 * j, djp + j * kRecordCols + kRecordTerm);
          tmem_copy(tmem + kTmJp + 64 + 8 * j, djp + kRecordThird / 16 + j * kRecordTerm);
        }
        if (!(ok = DELTA_WAIT(xready, c))) break;
        tc_fence_after();
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j) {  // [J; P~] X
          mma_ts(tmem + kTmSecond, tmem + kTmJp + 8 * j, dx + j * kTermStep, all, j > 0);
          mma_ts(tmem + kTmSecond, tmem + kTmJp + 32 + 8 * j, dx + j * kTermStep, less, true);
          mma_ts(tmem + kTmSecond, tmem + kTmJp + 64 + 8 * j, dx + j * kTermStep, one, true);
        }
        mma_commit(acc2);
        if (c + 1 < chunks) copy_kq(c + 1);
        if (!ok || !(ok = DELTA_WAIT(uready, c))) break;
        tc_fence_after();
        if (c + 1 < chunks || keep) {
          const uint64_t da = tile_desc(slot, kPanelBytes);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)  // K^T (eb . u)
            mma_ss(tmem + kTmThird, da + j * kKqRows, dx + j * kTermStep, last, j > 0);
          mma_commit(acc3);
        }
        mma_commit(empty + 8 * st);
      }
      // nothing of this CTA may be in flight when its shared memory and TMEM go
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (BWD && warp == 2) {
    // ---- two terms of every S_0 ----
    if (elect_one()) {
      for (int c = 0; c < chunks && ok; ++c) {
        if (!(ok = DELTA_WAIT(sready, c))) break;
        bulk_store(p.heads + (((slot0 + c) * p.Hv + w.hv) * p.tiles + w.tile) * 2 * kStatePanel, smem + kOffState,
                   2 * kStatePanel);
        stores_commit();
        stores_wait_read();
        bar_arrive(kept);
      }
      stores_wait();
    }
  } else if (warp >= 4 && warp < 4 + kRowWarps) {
    // ---- rows: 16 columns of a channel's state; pairs of columns of two tokens ----
    const int quarter = warp % 4, h = warp / 4 - 1;      // lanes of TMEM, half of the columns
    const int row = quarter * 32 + lane, col = col0 + h * 16, width = p.V - col;
    const int t = quarter * 16 + lane / 4;               // and t + 8
    const uint32_t mine = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + h * 16;
    const uint32_t other = mine + (static_cast<uint32_t>(kOther) << 16);
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
    put_terms8(smem + kOffState, kStatePanel, row, 2 * h, S);
    put_terms8(smem + kOffState, kStatePanel, row, 2 * h + 1, S + 8);
    cconv::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(sready);
    const uint16_t *v_at = p.v.p + w.hv * p.v.sh + col, *do_at = p.d_o.p + w.hv * p.d_o.sh + col;
    const int turned = quarter * 16 + quad_token(lane), turned_col = quad_column(lane);
    const bool inside = turned_col < width;
    uint32_t vw[2][2], dw[2][2];  // [token][columns] of v and do
    auto fetch = [&](int c) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t at = static_cast<int64_t>(w.a) + c * kDelta + t + 8 * r;
        load_words(at < w.b ? v_at + at * p.v.st : nullptr, width, lane, vw[r]);
        if (BWD) load_words(at < w.b ? do_at + at * p.d_o.st : nullptr, width, lane, dw[r]);
      }
    };
    fetch(0);
    for (int c = 0; c < chunks; ++c) {
      const int st = c & 1, row0 = w.a + c * kDelta, n = min(kDelta, w.b - row0);
      const float* gates = reinterpret_cast<const float*>(base + st * kSlotBytes + kSlotKq + kRecordGates);
      Pairs v, d;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          v.v[j][r] = bf16x2_to_f2(vw[r][j]);
          if (BWD) d.v[j][r] = bf16x2_to_f2(dw[r][j]);
        }
      fetch(c + 1);
      if (!(ok = DELTA_WARP_WAIT(rfull + 8 * st, c / 2))) break;
      float ef[2], eb[2], beta[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) ef[r] = gates[kEf + t + 8 * r], eb[r] = gates[kEb + t + 8 * r], beta[r] = gates[kBeta + t + 8 * r];
      const float total = gates[kTotal];
      if (!(ok = DELTA_WARP_WAIT(acc1, c))) break;
      tc_fence_after();
      Pairs y = load_sum<kTerms>(mine + kTmFirst), x;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v.v[j][r] = f2_fma(f2_splat(-ef[r]), y.v[j][r], v.v[j][r]);  // r
          if (t + 8 * r >= n) v.v[j][r] = 0;
          x.v[j][r] = f2_mul(f2_splat(beta[r]), v.v[j][r]);
        }
      put_pairs(smem + kOffX, t, h, lane, x);
      if (n < kDelta) zero_tokens(smem + st * kSlotBytes, panels, n, false, threadIdx.x - 128);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(xready);
      if (!(ok = DELTA_WARP_WAIT(acc2, c))) break;
      tc_fence_after();
      y = load_sum<kTerms>(mine + kTmSecond);
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          v.v[j][r] = f2_add(v.v[j][r], y.v[j][r]);  // z
          x.v[j][r] = f2_mul(f2_splat(eb[r] * beta[r]), v.v[j][r]);
          if (t + 8 * r >= n) x.v[j][r] = 0;
        }
      put_pairs(smem + kOffX, t, h, lane, x);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(uready);
      // what waits for nothing more: o, or o . do, z and u
      y = load_sum<kTerms>(other + kTmSecond);
      x = load_sum<kTerms>(other + kTmFirst);
      const int64_t at = ((slot0 + c) * p.Hv + w.hv) * p.tiles + w.tile;
      uint32_t words[4], second[4];
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const f2 o = f2_mul(f2_splat(p.scale), f2_fma(f2_splat(ef[r]), x.v[j][r], y.v[j][r]));
          if (BWD) {
            float a, b;
            cconv::f2_unpack(f2_mul(o, d.v[j][r]), a, b);
            sum[r] += a + b;
            f2 u = f2_mul(f2_splat(beta[r]), v.v[j][r]);
            if (t + 8 * r >= n) u = 0;
            words[2 * j + r] = f2_to_bf16x2(u);
            second[2 * j + r] = f2_to_bf16x2(f2_fma(bf16x2_to_f2(words[2 * j + r]), f2_splat(-1.f), u));
          } else {
            words[2 * j + r] = f2_to_bf16x2(o);
          }
        }
      if (BWD) {
        uint8_t* to = p.u + at * kUTile + term_piece(turned, 2 * h + turned_col / 8);
        *reinterpret_cast<uint4*>(to) = quad_words(words, lane);
        *reinterpret_cast<uint4*>(to + kTokenPanel) = quad_words(second, lane);
        ulonglong2* z = reinterpret_cast<ulonglong2*>(p.z + pairs_at(at, warp - 4, lane));
        z[0] = make_ulonglong2(v.v[0][0], v.v[0][1]);
        z[kPairsNext] = make_ulonglong2(v.v[1][0], v.v[1][1]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
          if (t + 8 * r < n && (lane & 3) == 0)
            p.dots[(static_cast<int64_t>(w.tile * 2 + h) * p.Hv + w.hv) * p.total + row0 + t + 8 * r] = sum[r];
        }
      } else {
        const uint4 o = quad_words(words, lane);
        if (turned < n && inside)
          *reinterpret_cast<uint4*>(p.o + (static_cast<int64_t>(row0 + turned) * p.Hv + w.hv) * p.V + col + turned_col) = o;
      }
      if (BWD && c > 0 && c % kAnchorChunks == 0) {
        float4* to = reinterpret_cast<float4*>(
            p.anchors + ((anchor_of(w.a, c) * p.Hv + w.hv) * p.tiles + w.tile) * kAnchorFloats + row * kColumns + h * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
      }
      if (c + 1 < chunks || keep) {
        float z[16];
        if (!(ok = DELTA_WARP_WAIT(acc3, c))) break;
        tc_fence_after();
        load_sum16(mine + kTmThird, z);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = row < p.K ? fmaf(total, S[i], z[i]) : 0.f;
        if (c + 1 < chunks) {
          if (BWD && !(ok = DELTA_WARP_WAIT(kept, c))) break;
          put_terms8(smem + kOffState, kStatePanel, row, 2 * h, S);
          put_terms8(smem + kOffState, kStatePanel, row, 2 * h + 1, S + 8);
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
  if (!ok) atomicOr(fault, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

inline int ctas(const DeltaCall& c) { return c.s.nseq * c.s.Hv * delta_tiles(c.s.V); }
inline int args_of(const DeltaCall& c, Args& a) {
  int rc = CCONV_OK;
  if (c.s.total > 0) {
    rc = bind_context();
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, 16);
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, 16);
    if (rc != CCONV_OK) return rc;
  }
  a.v = c.v, a.d_o = c.d_o;
  a.cu = c.cu, a.slots = c.slots, a.status = c.status, a.checked = c.checked;
  a.initial = c.initial, a.fin = c.fin;
  a.o = c.o;
  a.records = c.records;
  a.z = c.z, a.u = c.u, a.heads = c.heads, a.dots = c.odots, a.anchors = c.anchors;
  a.scale = c.scale;
  a.total = c.s.total, a.nseq = c.s.nseq, a.ratio = c.s.Hv / c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.tiles = delta_tiles(c.s.V);
  return CCONV_OK;
}

}  // namespace chain
}  // namespace cattn
