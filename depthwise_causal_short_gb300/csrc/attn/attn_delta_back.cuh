// attn_delta_back.cuh -- the gated delta rule's chain backwards: the gradient of the state.
//
// The CTAs, ring, terms and roles of attn_delta_chain.cuh, from a sequence's last chunk to its first.
// D, the gradient of the state at the chunk's end, is kept as S is there.  A chunk's products:
//   K D                                   -> r' = eb . (K D),  X = beta r'
//   J^T X;  P~^T do                       -> du = r' + J^T X + scale P~^T do,  dv = beta du
//   K^T (-ef . dv);  Q^T (scale ef . do)  -> D = total D + ..
// J and P~ are read from their records with the rows as the contraction; the products of their first terms lie
// in lanes 0 to 15 of each quarter, those of the second ones in lanes 16 to 31 (in place of Q D).  The products
// that have do in them wait for nothing of the chain: P~^T do is made a chunk ahead, while the rows work; four
// warps prepare do for them.
// Bound as that chain is: 395 us of the same 128 CTAs, 5800 cycles a chunk (the rows' part between the first two
// products 1400 of them, beside the next record's load); tensor cores 16 %, memory 30 %.  dv's second term takes 15 us
// of it.  K and Q copied to tensor memory as a first operand gained nothing here.
// It needs nothing of the chain of the states but for dbeta and the anchors: where SMs are free both run in one
// launch (BESIDE), and a kernel behind them makes those two.
// It leaves dv, a second term of it, two terms of every D, dbeta = du . z, v . dv, and at every kAnchorChunks-th
// chunk <S_0, D_0>.
#pragma once

#include <cudaTypedefs.h>

#include "attn_chunk_host.h"
#include "attn_delta.cuh"

namespace cattn {
namespace back {

constexpr int kThreads = (4 + kRowWarps + 4) * 32;
// shared memory, from a 1024-byte boundary: a ring of two slots of K, Q and a record without its third terms;
// these, the slots' pieces 2i and 2i + 1 in turn
constexpr int kSlot = kSlotKq + kRecordThird;
constexpr int kOffThird = 2 * kSlot;
constexpr int kOffD = kOffThird + 2 * kTermBytes;
constexpr int kOffDx = kOffD + kTerms * kStatePanel;      // X, then -ef . dv
constexpr int kOffDo = kOffDx + kTerms * kTokenPanel;     // scale ef . do
constexpr int kOffDoRaw = kOffDo + kTerms * kTokenPanel;  // do: two slots
constexpr int kOffBars = kOffDoRaw + 2 * kTokenPanel;
constexpr int kBytes = kOffBars + 24 * 8 + 1024;
static_assert(kBytes <= 232448, "shared memory of one CTA");
// columns of tensor memory: three accumulators of three terms, P~^T do; and what the third terms of P~ and J make
constexpr int kTmFirst = 0, kTmSecond = 96, kTmThird = 192, kTmDo = 288, kTmDoLast = 320, kTmLast = 352;

struct Args {
  CUtensorMap mq, mk;
  Rows v, d_o;
  const int32_t* cu;
  const uint8_t* records;
  const float* z;
  uint8_t* ends;          // [slots][Hv][tiles] two terms of D
  uint8_t* rest;          // [slots][Hv][tiles] what dv's rounding leaves, 64 rows of kColumns as the terms lie
  const float* anchors;   // [anchors][Hv][tiles]
  float* adots;           // [anchors][Hv][tiles * kRowWarps]
  float *du, *danchors;   // BESIDE: du as z is kept, D as the states are
  float *vdots, *bdots;   // [2 tiles][Hv][total]
  uint16_t* dv;
  float* dinit;
  float scale;
  int total, nseq, ratio, Hv, K, V, tiles;
};

// CTA `cta` of the chain.  BESIDE: the chain of the states runs at the same time; what needs both (dbeta and <S_0, D_0>)
// is left to the kernel behind.
template <bool BESIDE>
__device__ __forceinline__ void run(const Args& p, int cta, unsigned* fault) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t kfull = smem + kOffBars, rfull = kfull + 16, empty = rfull + 16, rawready = empty + 16;
  const uint32_t oready = rawready + 16, dready = oready + 8, xready = dready + 8, uready = xready + 8;
  const uint32_t acc1 = uready + 8, acc2 = acc1 + 8, acc3 = acc2 + 8;
  const uint32_t kept = acc3 + 8, alldone = kept + 8;
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(kfull + 8 * i, 1);
      bar_init(rfull + 8 * i, 1);
      bar_init(empty + 8 * i, 1 + kRowWarps + 4);
      bar_init(rawready + 8 * i, 4);
    }
    bar_init(oready, 4);
    bar_init(dready, kRowWarps);
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
  const int tile = cta % p.tiles;
  const int hv = cta / p.tiles % p.Hv;
  const int seq = cta / p.tiles / p.Hv;
  int row_a, row_b;
  sequence_rows(p.cu, seq, p.total, row_a, row_b);
  if (p.cu[seq] < 0 || p.cu[seq + 1] < p.cu[seq] || p.cu[seq + 1] > p.total) row_b = row_a;  // (reported already)
  const int chunks = (row_b - row_a + kDelta - 1) / kDelta;
  const int64_t slot0 = row_a / kDelta + seq;
  const int col0 = tile * kColumns, panels = p.K > kPanelCols ? 2 : 1;
  bool ok = true;

  if (warp == 0) {
    // ---- K, Q and records ----
    if (elect_one()) {
      const int hk = hv / p.ratio;
      int i = 0, part = 0;
      for (; i < chunks && ok; ++i) {
        const int st = i & 1, c = chunks - 1 - i;
        const uint32_t slot = smem + st * kSlot;
        if (i >= 2 && !(ok = DELTA_WAIT(empty + 8 * st, i / 2 - 1))) break;
        if (i > 0 && !(ok = DELTA_WAIT(acc1, i - 1))) break;
        // (the record first: P~^T do needs it, and before the chunk's other products)
        bar_expect(rfull + 8 * st, kRecordBytes);
        const uint8_t* record = p.records + ((slot0 + c) * p.Hv + hv) * kRecordBytes;
        bulk_load(slot + kSlotKq, record, kRecordThird, rfull + 8 * st);
#pragma unroll 1
        for (int j = 0; j < 4; ++j)
          bulk_load(smem + kOffThird + (2 * j + st) * 2 * kPieceBytes, record + kRecordThird + j * 2 * kPieceBytes,
                    2 * kPieceBytes, rfull + 8 * st);
        part = 1;
        if (i > 0 && !(ok = DELTA_WAIT(acc2, i - 1))) break;
        load_kq(slot, kfull + 8 * st, &p.mk, &p.mq, panels, hk, row_a + c * kDelta);
        part = 0;
      }
      for (int st = 0; st < 2; ++st) {
        drain(rfull + 8 * st, (i + part - st + 1) / 2);
        drain(kfull + 8 * st, (i - st + 1) / 2);
      }
    }
  } else if (warp == 1) {
    // ---- products ----
    if (elect_one()) {
      const int ksteps = (p.K + 15) / 16;
      const uint64_t dd = term_desc(smem + kOffD, kStatePanel), dx = term_desc(smem + kOffDx, kTokenPanel);
      const uint64_t dos = term_desc(smem + kOffDo, kTokenPanel);
      const uint32_t rows = mma_desc(3 * kColumns, false, true), three = mma_desc(3 * kColumns, true, true);
      const uint32_t one = mma_desc(kColumns, true, true);
      auto early = [&](int i) {  // P~^T do of chunk i
        const int st = i & 1;
        if (!(ok = DELTA_WAIT(rfull + 8 * st, i / 2)) || !(ok = DELTA_WAIT(rawready + 8 * st, i / 2))) return;
        tc_fence_after();
        const uint64_t dp = record_desc(smem + st * kSlot + kSlotKq + kOther * 16, true);
        const uint64_t from = term_desc(smem + kOffDoRaw + st * kTokenPanel, kTokenPanel);
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j)
          mma_ss(tmem + kTmDo, dp + j * kRecordRows, from + j * kTermStep, one, j > 0);
        // (third terms: lanes 16 to 31 of each quarter, the other slot's, are not read)
        const uint64_t third = record_desc(smem + kOffThird + st * 2 * kPieceBytes + kOther * 16, true);
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j)
          mma_ss(tmem + kTmDoLast, third + j * kRecordRows, from + j * kTermStep, one, j > 0);
      };
      if (chunks > 0) early(0);
      for (int i = 0; i < chunks && ok; ++i) {
        const int st = i & 1;
        const uint32_t slot = smem + st * kSlot;
        if (!(ok = DELTA_WAIT(kfull + 8 * st, i / 2))) break;
        if (!(ok = DELTA_WAIT(dready, i))) break;
        tc_fence_after();
        const uint64_t dkq = tile_desc(slot, 0);
#pragma unroll 1
        for (int j = 0; j < ksteps; ++j)  // K D
          mma_ss(tmem + kTmFirst, dkq + col_step(j), dd + j * kTermStep, rows, j > 0);
        mma_commit(acc1);
        if (!(ok = DELTA_WAIT(xready, i))) break;
        tc_fence_after();
        const uint64_t dj = record_desc(slot + kSlotKq, true);
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j)  // J^T X
          mma_ss(tmem + kTmSecond, dj + j * kRecordRows, dx + j * kTermStep, three, j > 0);
        const uint64_t third = record_desc(smem + kOffThird + st * 2 * kPieceBytes, true);
#pragma unroll 1
        for (int j = 0; j < kDelta / 16; ++j)
          mma_ss(tmem + kTmLast, third + j * kRecordRows, dx + j * kTermStep, one, j > 0);
        mma_commit(acc2);
        const bool more = i + 1 < chunks || p.dinit;
        if (!(ok = DELTA_WAIT(oready, i))) break;
        tc_fence_after();
        if (more) {
          const uint64_t da = tile_desc(slot + kOther * 128, kPanelBytes);  // Q^T (scale ef . do)
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem + kTmThird, da + j * kKqRows, dos + j * kTermStep, three, j > 0);
        }
        if (!(ok = DELTA_WAIT(uready, i))) break;
        tc_fence_after();
        if (more) {
          const uint64_t da = tile_desc(slot, kPanelBytes);  // K^T (-ef . dv)
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j)
            mma_ss(tmem + kTmThird, da + j * kKqRows, dx + j * kTermStep, three, true);
          mma_commit(acc3);
        }
        mma_commit(empty + 8 * st);
        if (i + 1 < chunks) early(i + 1);
      }
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (warp == 2) {
    // ---- two terms of every D, once K D does not read beside it ----
    if (elect_one()) {
      for (int i = 0; i < chunks && ok; ++i) {
        if (!(ok = DELTA_WAIT(dready, i)) || !(ok = DELTA_WAIT(acc1, i))) break;
        bulk_store(p.ends + (((slot0 + chunks - 1 - i) * p.Hv + hv) * p.tiles + tile) * 2 * kStatePanel, smem + kOffD,
                   2 * kStatePanel);
        stores_commit();
        stores_wait_read();
        bar_arrive(kept);
      }
      stores_wait();
    }
  } else if (warp >= 4 + kRowWarps) {
    // ---- do, as it is (a chunk ahead) and scaled: 16 columns of a token ----
    const int t = (warp & 1) * 32 + lane, half = (warp - 4 - kRowWarps) / 2;
    const int col = col0 + half * 16, width = p.V - col;
    const uint16_t* src = p.d_o.p + hv * p.d_o.sh + col;
    uint4 in[2];
    auto put_raw = [&](int i) {
      const int64_t at = static_cast<int64_t>(row_a) + (chunks - 1 - i) * kDelta + t;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        in[j] = make_uint4(0, 0, 0, 0);
        if (at < row_b && 8 * j < width) in[j] = *reinterpret_cast<const uint4*>(src + at * p.d_o.st + 8 * j);
        sts128(smem + kOffDoRaw + (i & 1) * kTokenPanel + term_piece(t, half * 2 + j), in[j].x, in[j].y, in[j].z, in[j].w);
      }
      cconv::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(rawready + 8 * (i & 1));
    };
    if (chunks > 0) put_raw(0);
    for (int i = 0; i < chunks; ++i) {
      const int st = i & 1;
      if (!(ok = DELTA_WARP_WAIT(rfull + 8 * st, i / 2))) break;
      const float f = p.scale * reinterpret_cast<const float*>(base + st * kSlot + kSlotKq + kRecordGates)[kEf + t];
      if (i > 0 && !(ok = DELTA_WARP_WAIT(acc3, i - 1))) break;  // the last chunk's are not needed any more
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x[8];
        unpack8(in[j], x);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= f;
        put_terms8(smem + kOffDo, kTokenPanel, t, half * 2 + j, x);
      }
      cconv::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(oready);
      if (lane == 0) bar_arrive(empty + 8 * st);
      // (P~^T do of chunk i - 1, the last reader of that slot, was done before its acc3)
      if (i + 1 < chunks) put_raw(i + 1);
    }
  } else if (warp >= 4) {
    // ---- rows: 16 columns of a channel of D; pairs of columns of two tokens ----
    const int quarter = warp % 4, h = warp / 4 - 1;
    const int row = quarter * 32 + lane, col = col0 + h * 16, width = p.V - col;
    const int t = quarter * 16 + lane / 4;
    const uint32_t mine = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + h * 16;
    const uint32_t other = mine + (static_cast<uint32_t>(kOther) << 16);
    float D[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i] = 0.f;
    put_terms8(smem + kOffD, kStatePanel, row, 2 * h, D);
    put_terms8(smem + kOffD, kStatePanel, row, 2 * h + 1, D + 8);
    cconv::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) bar_arrive(dready);
    const uint16_t* v_at = p.v.p + hv * p.v.sh + col;
    const int turned = quarter * 16 + quad_token(lane), turned_col = quad_column(lane);
    const bool inside = turned_col < width;
    uint32_t vw[2][2];
    Pairs zin;
    auto fetch = [&](int c) {
      if (c < 0) return;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t at = static_cast<int64_t>(row_a) + c * kDelta + t + 8 * r;
        load_words(at < row_b ? v_at + at * p.v.st : nullptr, width, lane, vw[r]);
      }
      if (BESIDE) return;
      const ulonglong2* z = reinterpret_cast<const ulonglong2*>(
          p.z + pairs_at(((slot0 + c) * p.Hv + hv) * p.tiles + tile, warp - 4, lane));
      const ulonglong2 a = z[0], b = z[kPairsNext];
      zin.v[0][0] = a.x, zin.v[0][1] = a.y, zin.v[1][0] = b.x, zin.v[1][1] = b.y;
    };
    fetch(chunks - 1);
    for (int i = 0; i < chunks; ++i) {
      const int st = i & 1, c = chunks - 1 - i, row0 = row_a + c * kDelta, n = min(kDelta, row_b - row0);
      const float* gates = reinterpret_cast<const float*>(base + st * kSlot + kSlotKq + kRecordGates);
      Pairs v, z;
      if (!BESIDE) z = zin;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 2; ++r) v.v[j][r] = bf16x2_to_f2(vw[r][j]);
      fetch(c - 1);
      const bool anchor = c > 0 && c % kAnchorChunks == 0;
      const int64_t anchor_at = (anchor_of(row_a, c) * p.Hv + hv) * p.tiles + tile;
      const float* state = p.anchors + anchor_at * kAnchorFloats + row * kColumns + h * 16;
      if (anchor && !BESIDE) asm volatile("prefetch.global.L2 [%0];" ::"l"(state));
      if (!(ok = DELTA_WARP_WAIT(rfull + 8 * st, i / 2))) break;
      float ef[2], eb[2], beta[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) ef[r] = gates[kEf + t + 8 * r], eb[r] = gates[kEb + t + 8 * r], beta[r] = gates[kBeta + t + 8 * r];
      const float total = gates[kTotal];
      if (!(ok = DELTA_WARP_WAIT(acc1, i))) break;
      tc_fence_after();
      Pairs y = load_sum<3>(mine + kTmFirst), x;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          y.v[j][r] = f2_mul(f2_splat(eb[r]), y.v[j][r]);  // r'
          if (t + 8 * r >= n) y.v[j][r] = 0;
          x.v[j][r] = f2_mul(f2_splat(beta[r]), y.v[j][r]);
        }
      put_pairs(smem + kOffDx, t, h, lane, x);
      if (n < kDelta) zero_tokens(smem + st * kSlot, panels, n, true, threadIdx.x - 128);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(xready);
      if (!(ok = DELTA_WARP_WAIT(acc2, i))) break;
      tc_fence_after();
      {
        Pairs first = load_sum<3>(mine + kTmSecond), second = load_sum<3>(other + kTmSecond);
        const Pairs a = load_sum<2>(mine + kTmDo), b = load_sum<1>(other + kTmDo), last = load_sum<1>(mine + kTmLast);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const f2 from_do = f2_mul(f2_splat(p.scale), f2_add(a.v[j][r], b.v[j][r]));
            second.v[j][r] = f2_add(second.v[j][r], last.v[j][r]);
            y.v[j][r] = f2_add(y.v[j][r], f2_add(from_do, f2_add(first.v[j][r], second.v[j][r])));  // du
            if (t + 8 * r >= n) y.v[j][r] = 0;
            x.v[j][r] = f2_mul(f2_splat(-ef[r] * beta[r]), y.v[j][r]);
          }
      }
      put_pairs(smem + kOffDx, t, h, lane, x);
      cconv::fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(uready);
      uint32_t words[4], second[4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float du_z = 0.f, dv_v = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const f2 dv = f2_mul(f2_splat(beta[r]), y.v[j][r]);
          float a, b;
          if (!BESIDE) {
            cconv::f2_unpack(f2_mul(y.v[j][r], z.v[j][r]), a, b);
            du_z += a + b;
          }
          cconv::f2_unpack(f2_mul(dv, v.v[j][r]), a, b);
          dv_v += a + b;
          words[2 * j + r] = f2_to_bf16x2(dv);
          second[2 * j + r] = f2_to_bf16x2(f2_fma(bf16x2_to_f2(words[2 * j + r]), f2_splat(-1.f), dv));
        }
        if (!BESIDE) du_z += __shfl_xor_sync(0xffffffffu, du_z, 1);
        dv_v += __shfl_xor_sync(0xffffffffu, dv_v, 1);
        if (!BESIDE) du_z += __shfl_xor_sync(0xffffffffu, du_z, 2);
        dv_v += __shfl_xor_sync(0xffffffffu, dv_v, 2);
        if (t + 8 * r < n && (lane & 3) == 0) {
          const int64_t at = (static_cast<int64_t>(tile * 2 + h) * p.Hv + hv) * p.total + row0 + t + 8 * r;
          if (!BESIDE) p.bdots[at] = du_z;
          p.vdots[at] = dv_v;
        }
      }
      if (BESIDE) {
        ulonglong2* du = reinterpret_cast<ulonglong2*>(
            p.du + pairs_at(((slot0 + c) * p.Hv + hv) * p.tiles + tile, warp - 4, lane));
        du[0] = make_ulonglong2(y.v[0][0], y.v[0][1]);
        du[kPairsNext] = make_ulonglong2(y.v[1][0], y.v[1][1]);
      }
      *reinterpret_cast<uint4*>(p.rest + (((slot0 + c) * p.Hv + hv) * p.tiles + tile) * kTokenPanel +
                                term_piece(turned, 2 * h + turned_col / 8)) = quad_words(second, lane);
      const uint4 dv = quad_words(words, lane);
      if (turned < n && inside)
        *reinterpret_cast<uint4*>(p.dv + (static_cast<int64_t>(row0 + turned) * p.Hv + hv) * p.V + col + turned_col) = dv;
      if (i + 1 < chunks || p.dinit) {
        float g[16];
        if (!(ok = DELTA_WARP_WAIT(acc3, i))) break;
        tc_fence_after();
        load_sum16(mine + kTmThird, g);
#pragma unroll
        for (int j = 0; j < 16; ++j) D[j] = row < p.K ? fmaf(total, D[j], g[j]) : 0.f;
        if (i + 1 < chunks) {
          if (!(ok = DELTA_WARP_WAIT(kept, i))) break;
          put_terms8(smem + kOffD, kStatePanel, row, 2 * h, D);
          put_terms8(smem + kOffD, kStatePanel, row, 2 * h + 1, D + 8);
          cconv::fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(dready);
          if (BESIDE && anchor) {
            float4* to = reinterpret_cast<float4*>(p.danchors + (state - p.anchors));
#pragma unroll
            for (int j = 0; j < 4; ++j) to[j] = make_float4(D[4 * j], D[4 * j + 1], D[4 * j + 2], D[4 * j + 3]);
          } else if (anchor) {
            const float4* s = reinterpret_cast<const float4*>(state);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += dot4(make_float4(D[4 * j], D[4 * j + 1], D[4 * j + 2], D[4 * j + 3]), s[j]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) p.adots[anchor_at * kRowWarps + warp - 4] = sum;
          }
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
  if (!ok) atomicOr(fault, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

inline int args_of(const DeltaCall& c, Args& a) {
  int rc = bind_context();
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, 16);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, 16);
  if (rc != CCONV_OK) return rc;
  a.v = c.v, a.d_o = c.d_o;
  a.cu = c.cu;
  a.records = c.records;
  a.z = c.z;
  a.ends = c.ends, a.rest = c.rest;
  a.anchors = c.anchors, a.adots = c.adots;
  a.du = c.du, a.danchors = c.danchors;
  a.vdots = c.vdots, a.bdots = c.bdots;
  a.dv = c.dv, a.dinit = c.dinit;
  a.scale = c.scale;
  a.total = c.s.total, a.nseq = c.s.nseq, a.ratio = c.s.Hv / c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.tiles = delta_tiles(c.s.V);
  return CCONV_OK;
}

}  // namespace back
}  // namespace cattn
