// attn_delta_grads.cu -- the gated delta rule's dq and dk, and the sums that give dg and dbeta.
//
// With S_0 and D, the state before a chunk and the gradient of the state behind it, known (the chains
// left two bf16 terms of them, and of u), all chunks are done at once; per chunk and value head
//   X = scale (do u^T) . L (s <= t),   Y = (dv u^T) . L (s < t)
//   dq = X K                        + scale ef . (do S_0^T)
//   dk = X^T Q - (Y + Y^T) K + eb . (u D^T) - ef . (dv S_0^T)
// summed over the value heads of a key head in the CTA's registers.  do and dv lie one over the other
// as a first operand of 128 rows, and so do dq and dk as results:
//   [do; dv] u^T,  [0; dv'] u^T              -> X, -Y
//   [do; dv] S_0^T,  [0; dv'] S_0^T          rows scaled by scale ef and -ef afterwards
//   [  ; u ] D^T                             rows 64.. scaled by eb afterwards
//   [X; -Y] K,  [0; -Y^T] K,  [0; X^T] Q
// A CTA goes through (chunk, key head) items; do, dv, u and the tiles of S_0 and D come by TMA, 32 columns
// of V at a time, through a ring for what X and Y need and one for the states.  Every factor that is no input keeps
// two terms, dv as it is stored and what that leaves (dv'): 16 bits, for results of 9.  With all of them in one term
// dk's error in the 2-norm was 2.8e-3, with dv alone 1.8e-3 to 2.1e-3; the store makes 1.7e-3.
// Bound by memory, and the loads' latency behind it: 209 us for 16384 rows of 16 heads on 8 of 128 x 128, 1032 MB
// (4.9 TB/s, 73 % of a copy's rate), of which two terms of S_0 and of D are 537.  One CTA an SM (212 KB).
#include <cudaTypedefs.h>

#include "attn_chunk_host.h"
#include "attn_delta.cuh"

namespace cattn {

static __device__ unsigned g_fault_grads;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_grads, sizeof(*out))) != cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_grads, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

// shared memory, from a 1024-byte boundary
constexpr int kHalf = kDelta * 128;                       // 64 rows of 64 columns
// do over dv; two terms of u; zeros over dv'
constexpr int kPairDv = kTokenPanel, kPairU = 2 * kTokenPanel, kPairRest = kPairU + kUTile;
constexpr int kPairLoads = kPairRest + kTokenPanel, kPairSlot = kPairRest + 2 * kTokenPanel;
constexpr int kStateSlot = 4 * kStatePanel;               // two terms of S_0 and of D
constexpr int kPairSlots = 3, kStateSlots = 2;
constexpr int kOffStates = kPairSlots * kPairSlot;
constexpr int kOffGradKq = kOffStates + kStateSlots * kStateSlot;
constexpr int kOffZero = kOffGradKq + kSlotKq;           // zeros; X, -Y; their second terms: 64 rows each
constexpr int kOffXy = kOffZero + kHalf;
constexpr int kOffGates = kOffXy + 4 * kHalf;             // of two heads in turn
constexpr int kHeadGates = 5 * kDelta;                    // floats
constexpr int kOffGradBars = kOffGates + 2 * kHeadGates * 4;
constexpr int kGradBytes = kOffGradBars + 24 * 8 + 1024;
static_assert(kGradBytes <= 232448, "shared memory of one CTA");
// columns of TMEM
constexpr int kAccXy = 0, kAccState = 128, kAccEnd = 256, kAccIntra = 384;  // X, Y: two heads in turn
constexpr int kPartsAhead = 8;  // parts of the sums in flight
constexpr int kGradThreads = 384, kGradRowWarps = 8;

struct GradArgs {
  CUtensorMap mq, mk, mo, mv;  // q, k; do, dv in boxes of 32 columns
  Gates g;
  const int32_t* cu;
  const uint8_t *u, *heads, *ends, *rest;
  const float *odots, *vdots, *bdots;
  uint16_t *dq, *dk;
  float *dg, *dbeta;
  double* sums;  // [Hv][slots], see DeltaCall
  int* shut;
  float scale;
  int total, nseq, Hk, Hv, K, V, tiles, fresh;
  int64_t items;  // slots * Hk
};

__global__ void __launch_bounds__(kGradThreads, 1) cattn_delta_grads_kernel(const __grid_constant__ GradArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t pfull = smem + kOffGradBars, pempty = pfull + 8 * kPairSlots;    // do, dv, u of a tile
  const uint32_t sfull = pempty + 8 * kPairSlots, sempty = sfull + 8 * kStateSlots;  // its states
  const uint32_t kqfull = sempty + 8 * kStateSlots, kqempty = kqfull + 8;          // an item's K and Q
  const uint32_t xyfull = kqempty + 8, xyready = xyfull + 8;                      // a head's X and Y
  const uint32_t headfull = xyready + 8, headfree = headfull + 8;                 // a head's sums
  const uint32_t gready = headfree + 8, gfree = gready + 16, alldone = gfree + 16;  // a head's gates, in turn
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ratio = p.Hv / p.Hk;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairSlots; ++i) {
      bar_init(pfull + 8 * i, 1);
      bar_init(pempty + 8 * i, 1);
    }
    for (int i = 0; i < kStateSlots; ++i) {
      bar_init(sfull + 8 * i, 1);
      bar_init(sempty + 8 * i, 1);
    }
    bar_init(kqfull, 1);
    bar_init(kqempty, 1);
    bar_init(xyfull, 1);
    bar_init(xyready, kGradRowWarps);
    bar_init(headfull, 1);
    bar_init(headfree, kGradRowWarps);
    for (int i = 0; i < 2; ++i) {
      bar_init(gready + 8 * i, 1);
      bar_init(gfree + 8 * i, kGradRowWarps);
    }
    bar_init(alldone, 1);
    cconv::fence_mbar_init();
  }
  for (int i = threadIdx.x; i < kHalf / 16; i += kGradThreads) sts128(smem + kOffZero + i * 16, 0, 0, 0, 0);
  for (int i = threadIdx.x; i < kPairSlots * kTokenPanel / 16; i += kGradThreads)
    sts128(smem + i / (kTokenPanel / 16) * kPairSlot + kPairRest + i % (kTokenPanel / 16) * 16, 0, 0, 0, 0);
  cconv::fence_proxy_async_smem();
  if (warp == 1) tmem_alloc(&tmem_at, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  bool ok = true;

  if (warp == 0) {
    // ---- tiles ----
    int pairs = 0, states = 0, item = 0, part = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      const int hk = static_cast<int>(at % p.Hk);
      const int64_t slot = at / p.Hk;
      Chunk x;
      if (!find_chunk(p.cu, p.nseq, p.total, slot, lane, x)) continue;
      if (elect_one()) {
        const int panels = p.K > kPanelCols ? 2 : 1;
        if (item > 0) ok = DELTA_WAIT(kqempty, item - 1);
        if (ok) {
          bar_expect(kqfull, panels * 2 * kSideBytes);
          for (int j = 0; j < panels; ++j) {
            load_box(smem + kOffGradKq + j * kPanelBytes, &p.mk, kqfull, j * kPanelCols, hk, x.row0);
            load_box(smem + kOffGradKq + j * kPanelBytes + kSideBytes, &p.mq, kqfull, j * kPanelCols, hk, x.row0);
          }
          part = 1;
        }
        for (int h = 0; h < ratio && ok; ++h) {
          const int hv = hk * ratio + h;
          const int64_t first = (slot * p.Hv + hv) * p.tiles;
          // states follow the pairs as the products take them (below)
          int done = 0;
          auto load_states = [&](int end) {
            for (; done < end && ok; ++done, ++states) {
              const int st = states % kStateSlots;
              if (states >= kStateSlots && !(ok = DELTA_WAIT(sempty + 8 * st, states / kStateSlots - 1))) return;
              const uint32_t dst = smem + kOffStates + st * kStateSlot, bar = sfull + 8 * st;
              bar_expect(bar, kStateSlot);
              bulk_load(dst, p.heads + (first + done) * 2 * kStatePanel, 2 * kStatePanel, bar);
              bulk_load(dst + 2 * kStatePanel, p.ends + (first + done) * 2 * kStatePanel, 2 * kStatePanel, bar);
            }
          };
          for (int s = 0; s < p.tiles && ok; ++s, ++pairs) {
            const int st = pairs % kPairSlots;
            if (pairs >= kPairSlots && !(ok = DELTA_WAIT(pempty + 8 * st, pairs / kPairSlots - 1))) break;
            const uint32_t dst = smem + st * kPairSlot, bar = pfull + 8 * st;
            bar_expect(bar, kPairLoads);
            load_box(dst, &p.mo, bar, s * kColumns, hv, x.row0);
            load_box(dst + kPairDv, &p.mv, bar, s * kColumns, hv, x.row0);
            bulk_load(dst + kPairU, p.u + (first + s) * kUTile, kUTile, bar);
            bulk_load(dst + kPairRest + kTokenPanel, p.rest + (first + s) * kTokenPanel, kTokenPanel, bar);
            if (s + 1 == p.tiles)
              load_states(p.tiles);
            else if (s + 1 >= kPairSlots)
              load_states(s + 2 - kPairSlots);
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      pairs = __reduce_max_sync(0xffffffffu, pairs);
      states = __reduce_max_sync(0xffffffffu, states);
      if (ok) ++item, part = 0;
    }
    item += __any_sync(0xffffffffu, part);
    if (elect_one()) {
      drain(kqfull, item);
      // (a pair's or state's loads that gave up half-way count where they were begun)
      for (int st = 0; st < kPairSlots; ++st) drain(pfull + 8 * st, (pairs - st + kPairSlots - 1) / kPairSlots);
      for (int st = 0; st < kStateSlots; ++st) drain(sfull + 8 * st, (states - st + kStateSlots - 1) / kStateSlots);
    }
  } else if (warp == 1) {
    // ---- products ----
    int pairs = 0, states = 0, item = 0, head = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      Chunk x;
      if (!find_chunk(p.cu, p.nseq, p.total, at / p.Hk, lane, x)) continue;
      if (elect_one()) {
        const int width = p.K > kPanelCols ? 128 : 64;  // channels of the results
        const uint32_t d_xy = mma_desc(kDelta, false, false), d_state = mma_desc(width, false, false);
        const uint32_t d_rows = mma_desc(width, false, true), d_cols = mma_desc(width, true, true);
        ok = DELTA_WAIT(kqfull, item);
        for (int h = 0; h < ratio && ok; ++h, ++head) {
          const uint32_t xy_acc = tmem + kAccXy + (head & 1) * kDelta;
          // X and Y of as many tiles as there are slots, then the products with the states of one for each
          // further one, and of those that are left
          int done = 0;
          auto with_states = [&](int end) {
            if (done == 0 && head > 0 && !(ok = DELTA_WAIT(headfree, head - 1))) return;
            for (; done < end && ok; ++done, ++states) {
              const int at_pair = (pairs + done) % kPairSlots, at_state = states % kStateSlots;
              if (!(ok = DELTA_WAIT(sfull + 8 * at_state, states / kStateSlots))) return;
              tc_fence_after();
              const uint32_t pair = smem + at_pair * kPairSlot;
              const uint32_t state = smem + kOffStates + at_state * kStateSlot;
              const int ks = (min(kColumns, p.V - kColumns * done) + 15) / 16;
#pragma unroll 1
              for (int j = 0; j < ks; ++j) {
                const uint64_t rows = term_desc(pair, 0) + 2 * j, rest = rows + kPairRest / 16;
                const uint64_t start = term_desc(state, 0) + 2 * j, end = start + 2 * kStatePanel / 16;
                mma_ss(tmem + kAccState, rows, start, d_state, done + j > 0);
                mma_ss(tmem + kAccState, rows, start + kStatePanel / 16, d_state, true);
                mma_ss(tmem + kAccState, rest, start, d_state, true);
                const uint64_t first = rows + kPairDv / 16, second = rows + kPairU / 16;  // rows 64 on: terms of u
                mma_ss(tmem + kAccEnd, first, end, d_state, done + j > 0);
                mma_ss(tmem + kAccEnd, first, end + kStatePanel / 16, d_state, true);
                mma_ss(tmem + kAccEnd, second, end, d_state, true);
              }
              mma_commit(pempty + 8 * at_pair);
              mma_commit(sempty + 8 * at_state);
            }
          };
          for (int s = 0; s < p.tiles && ok; ++s) {
            const int st = (pairs + s) % kPairSlots;
            const uint32_t pair = smem + st * kPairSlot;
            const int ks = (min(kColumns, p.V - kColumns * s) + 15) / 16;
            if (!(ok = DELTA_WAIT(pfull + 8 * st, (pairs + s) / kPairSlots))) break;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < ks; ++j) {
              const uint64_t a = term_desc(pair, 0) + 2 * j, u = a + kPairU / 16;
              mma_ss(xy_acc, a, u, d_xy, s + j > 0);
              mma_ss(xy_acc, a, u + kTokenPanel / 16, d_xy, true);
              mma_ss(xy_acc, a + kPairRest / 16, u, d_xy, true);
            }
            if (s + 1 == p.tiles) {
              mma_commit(xyfull);
              with_states(p.tiles);
            } else if (s + 1 >= kPairSlots) {
              with_states(s + 2 - kPairSlots);
            }
          }
          pairs += p.tiles;
          if (!ok || !(ok = DELTA_WAIT(xyready, head))) break;
          tc_fence_after();
          const uint64_t k = tile_desc(smem + kOffGradKq, kPanelBytes);
          const uint64_t q = tile_desc(smem + kOffGradKq + kSideBytes, kPanelBytes);
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {  // first and second terms
            const uint64_t xy = tile_desc(smem + kOffXy + i * 2 * kHalf, 0);
            const uint64_t xt = tile_desc(smem + kOffZero, (1 + 2 * i) * kHalf);
            const uint64_t yt = tile_desc(smem + kOffZero, (2 + 2 * i) * kHalf);
#pragma unroll 1
            for (int j = 0; j < kDelta / 16; ++j) {
              mma_ss(tmem + kAccIntra, xy + 2 * j, k + j * kRowStep, d_rows, h + i + j > 0);
              mma_ss(tmem + kAccIntra, yt + j * kRowStep, k + j * kRowStep, d_cols, true);
              mma_ss(tmem + kAccIntra, xt + j * kRowStep, q + j * kRowStep, d_cols, true);
            }
          }
          mma_commit(headfull);
        }
        if (ok) mma_commit(kqempty);
      }
      ok = __all_sync(0xffffffffu, ok);
      pairs = __reduce_max_sync(0xffffffffu, pairs);
      states = __reduce_max_sync(0xffffffffu, states);
      head = __reduce_max_sync(0xffffffffu, head);
      ++item;
    }
    if (elect_one()) {
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (warp == 2) {
    // ---- dbeta, and dg summed up from each token to its chunk's end, or to the next shut gate ----
    for (int64_t at = blockIdx.x; at < p.items; at += gridDim.x) {
      const int64_t slot = at / p.Hk;
      Chunk chunk;
      if (!find_chunk(p.cu, p.nseq, p.total, slot, lane, chunk)) continue;
      const int row0 = chunk.row0, n = chunk.n;
      for (int h = 0; h < ratio; ++h) {
        const int hv = static_cast<int>(at % p.Hk) * ratio + h;
        double x[2] = {0.0, 0.0};
        float db[2] = {0.f, 0.f};
        bool shut[2];  // of tokens 63 - 2 lane, 62 - 2 lane; the first gate on no state counts as shut
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = kDelta - 1 - 2 * lane - j;
          shut[j] = t < n && ((p.fresh && row0 + t == chunk.a) || exp2_fast(kLog2e * p.g.at(row0 + t, hv)) == 0.f);
        }
        for (int first = 0; first < 2 * p.tiles; first += kPartsAhead) {
          float o[kPartsAhead][2], v[kPartsAhead][2], d[kPartsAhead][2];
#pragma unroll
          for (int i = 0; i < kPartsAhead; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int t = kDelta - 1 - 2 * lane - j;
              const int64_t from = (static_cast<int64_t>(first + i) * p.Hv + hv) * p.total + row0 + t;
              o[i][j] = v[i][j] = d[i][j] = 0.f;
              if (t < n && first + i < 2 * p.tiles) o[i][j] = p.odots[from], v[i][j] = p.vdots[from], d[i][j] = p.bdots[from];
            }
#pragma unroll
          for (int i = 0; i < kPartsAhead; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              x[j] += static_cast<double>(o[i][j]) - static_cast<double>(v[i][j]);
              db[j] += d[i][j];
            }
        }
        // the sum from a token on: 0 where its gate is shut
        double up = shut[1] ? 0.0 : shut[0] ? x[1] : x[0] + x[1];
        int cut = shut[0] | shut[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xffffffffu, up, o);
          const int before = __shfl_up_sync(0xffffffffu, cut, o);
          if (lane >= o) {
            if (!cut) up += y;
            cut |= before;
          }
        }
        const double behind = __shfl_up_sync(0xffffffffu, up, 1);
        const double sum0 = shut[0] ? 0.0 : lane > 0 ? x[0] + behind : x[0];
        const double sum1 = shut[1] ? 0.0 : x[1] + sum0;
        const float sums[2] = {static_cast<float>(sum0), static_cast<float>(sum1)};
        const int last = shut[0] ? kDelta - 1 - 2 * lane : shut[1] ? kDelta - 2 - 2 * lane : -1;
        const int last_shut = __reduce_max_sync(0xffffffffu, last);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int t = kDelta - 1 - 2 * lane - j;
          if (t >= n) continue;
          p.dbeta[static_cast<int64_t>(row0 + t) * p.Hv + hv] = db[j];
          p.dg[static_cast<int64_t>(row0 + t) * p.Hv + hv] = sums[j];
        }
        if (lane == 31) {
          p.sums[hv * (p.items / p.Hk) + slot] = sum1;
          p.shut[hv * (p.items / p.Hk) + slot] = last_shut;
        }
      }
    }
  } else if (warp == 3) {
    // ---- the heads' gates, two ahead ----
    int head = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      Chunk chunk;
      if (!find_chunk(p.cu, p.nseq, p.total, at / p.Hk, lane, chunk)) continue;
      const int row0 = chunk.row0, n = chunk.n;
      for (int h = 0; h < ratio; ++h, ++head) {
        const int hv = static_cast<int>(at % p.Hk) * ratio + h;
        float g[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) g[j] = 2 * lane + j < n ? kLog2e * p.g.at(row0 + 2 * lane + j, hv) : 0.f;
        // sums of one sign: within the block of 32 tokens (16 lanes), then with the other block
        const float own = g[0] + g[1];
        float up = own, down = own;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) {
          const float x = __shfl_up_sync(0xffffffffu, up, o, 16), y = __shfl_down_sync(0xffffffffu, down, o, 16);
          if ((lane & 15) >= o) up += x;
          if ((lane & 15) + o < 16) down += y;
        }
        const float first = __shfl_sync(0xffffffffu, down, 0), second = __shfl_sync(0xffffffffu, down, 16);
        float before = __shfl_up_sync(0xffffffffu, up, 1, 16), after = __shfl_down_sync(0xffffffffu, down, 1, 16);
        if ((lane & 15) == 0) before = 0.f;
        if ((lane & 15) == 15) after = 0.f;
        const float front = lane < 16 ? 0.f : first, rest = lane < 16 ? second : 0.f;
        if (head > 1 && !(ok = DELTA_WARP_WAIT(gfree + 8 * (head & 1), head / 2 - 1))) break;
        float2* to = reinterpret_cast<float2*>(base + kOffGates) + (head & 1) * (kHeadGates / 2) + lane;
        to[0] = make_float2(exp2_fast(g[0]), exp2_fast(g[1]));                                   // of the token
        to[32] = make_float2(exp2_fast(before + g[0]), exp2_fast(before + own));                 // from the block's start
        to[64] = make_float2(exp2_fast(g[1] + after), exp2_fast(after));                         // to its end
        to[96] = make_float2(exp2_fast(front + before + g[0]), exp2_fast(front + before + own)); // from the chunk's start
        to[128] = make_float2(exp2_fast(g[1] + after + rest), exp2_fast(after + rest));          // to its end
        __syncwarp();
        if (lane == 0) bar_arrive(gready + 8 * (head & 1));
      }
    }
  } else if (warp >= 4) {
    // ---- rows ----
    const int quarter = warp % 4, half = warp / 4 - 1;
    const int row = quarter * 32 + lane, t = row & (kDelta - 1), block = quarter & 1;
    const bool dq = quarter < 2;  // this thread's row is one of dq; or of dk
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int tid = threadIdx.x - 128;
    int item = 0, head = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      const int hk = static_cast<int>(at % p.Hk);
      Chunk chunk;
      if (!find_chunk(p.cu, p.nseq, p.total, at / p.Hk, lane, chunk)) continue;
      const int row0 = chunk.row0, n = chunk.n;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      for (int h = 0; h < ratio && ok; ++h, ++head) {
        const float* gates = reinterpret_cast<const float*>(base + kOffGates) + (head & 1) * kHeadGates;
        if (h == 0) {
          if (!(ok = DELTA_WARP_WAIT(kqfull, item))) break;
          if (n < kDelta) {
            // rows of the next sequence must not meet X, Y
            const int pieces = (kDelta - n) * 8, panels = p.K > kPanelCols ? 2 : 1;
            for (int e = tid; e < 2 * panels * pieces; e += 256) {
              const int side = e / pieces, i = e % pieces;
              sts128(smem + kOffGradKq + (side >> 1) * kPanelBytes + (side & 1) * kSideBytes + (n + i / 8) * 128 + (i % 8) * 16,
                     0, 0, 0, 0);
            }
          }
        }
        if (!(ok = DELTA_WARP_WAIT(gready + 8 * (head & 1), head / 2))) break;
        if (!(ok = DELTA_WARP_WAIT(xyfull, head))) break;
        tc_fence_after();
        {
          // columns s of block `half` times the decay from s to t: across blocks a product of two factors,
          // in the block itself a running product down from t
          float x[32];
          if (half <= block) {
            uint32_t y[32];
            tmem_ld32(tmem + lanes + kAccXy + (head & 1) * kDelta + half * 32, y);
            tmem_wait_ld();
            tmem_use32(y);
            const float f = t < n ? (dq ? p.scale : -1.f) : 0.f;
            if (half < block) {
              const float u = f * gates[64 + t];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 w = *reinterpret_cast<const float4*>(gates + 128 + 4 * i);
                x[4 * i] = u * w.x * __uint_as_float(y[4 * i]);
                x[4 * i + 1] = u * w.y * __uint_as_float(y[4 * i + 1]);
                x[4 * i + 2] = u * w.z * __uint_as_float(y[4 * i + 2]);
                x[4 * i + 3] = u * w.w * __uint_as_float(y[4 * i + 3]);
              }
            } else {
              float w = f;
#pragma unroll
              for (int i = 7; i >= 0; --i) {
                const float4 a = *reinterpret_cast<const float4*>(gates + half * 32 + 4 * i);
#pragma unroll
                for (int j = 3; j >= 0; --j) {
                  const int s = 4 * i + j;
                  x[s] = s < lane || (dq && s == lane) ? __uint_as_float(y[s]) * w : 0.f;
                  if (s <= lane) w *= j == 3 ? a.w : j == 2 ? a.z : j == 1 ? a.y : a.x;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = t < n ? x[i] : 0.f;
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f2 v = f2_pack(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
              hi[j] = f2_to_bf16x2(v);
              lo[j] = f2_to_bf16x2(f2_fma(bf16x2_to_f2(hi[j]), f2_splat(-1.f), v));
            }
            const uint32_t to = smem + kOffXy + swizzled(row, half * 4 + i);
            sts128(to, hi[0], hi[1], hi[2], hi[3]);
            sts128(to + 2 * kHalf, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        cconv::fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(xyready);
        const float ef = gates[192 + t], eb = gates[256 + t], f = dq ? p.scale * ef : -ef;
        __syncwarp();
        if (lane == 0) bar_arrive(gfree + 8 * (head & 1));
        if (!(ok = DELTA_WARP_WAIT(headfull, head))) break;
        tc_fence_after();
        const bool last = h + 1 == ratio;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int c = half * 64 + b * 16;
          if (c >= p.K) continue;
          uint32_t x[16], y[16], w[16];
          tmem_ld16(tmem + lanes + kAccState + c, x);
          if (!dq) tmem_ld16(tmem + lanes + kAccEnd + c, y);
          if (last) tmem_ld16(tmem + lanes + kAccIntra + c, w);
          tmem_wait_ld();
          tmem_use16(x);
          if (!dq) tmem_use16(y);
          if (last) tmem_use16(w);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float v = fmaf(f, __uint_as_float(x[i]), acc[b * 16 + i]);
            if (!dq) v = fmaf(eb, __uint_as_float(y[i]), v);
            if (last) v += __uint_as_float(w[i]);
            acc[b * 16 + i] = v;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(headfree);
      }
      if (!ok) break;
      ++item;
      if (t < n) {
        uint16_t* dst = (dq ? p.dq : p.dk) + (static_cast<int64_t>(row0 + t) * p.Hk + hk) * p.K + half * 64;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (half * 64 + 8 * i < p.K) *reinterpret_cast<uint4*>(dst + 8 * i) = pack8(acc + 8 * i);
      }
    }
  }
  if (!ok) atomicOr(&g_fault_grads, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// dg, second part: what the chunks behind a token's add, to the next shut gate, anchor or the sequence's end.  A CTA
// for each chunk, a warp for each value head in turn; kept in 64 bits, since terms of both signs cancel.
struct GateArgs {
  const int32_t* cu;
  const double* sums;
  const int* shut;
  const float* adots;
  float* dg;
  int total, nseq, Hv, parts;  // parts of an anchor
  int64_t slots;
};
constexpr int kGateThreads = 256;
__global__ void __launch_bounds__(kGateThreads) cattn_delta_gates_kernel(const GateArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ double later[kGateThreads];
  __shared__ int shut[kGateThreads];  // the last token of this chunk whose gate is shut
  const int lane = threadIdx.x % 32;
  Chunk x;
  const int64_t slot = blockIdx.x;
  if (!find_chunk(p.cu, p.nseq, p.total, slot, lane, x)) return;
  const int chunks = (x.b - x.a + kDelta - 1) / kDelta, next = (x.c / kAnchorChunks + 1) * kAnchorChunks;
  float* dg = p.dg + static_cast<int64_t>(x.row0) * p.Hv;
  for (int first = 0; first < p.Hv; first += kGateThreads) {
    const int heads = min(kGateThreads, p.Hv - first);
    for (int i = threadIdx.x / 32; i < heads; i += kGateThreads / 32) {
      const int hv = first + i;
      // (the chunks up to the next anchor are fewer than 32)
      const bool in = x.c + 1 + lane < min(next, chunks);
      const int64_t at = hv * p.slots + slot + 1 + lane;
      const unsigned cuts = __ballot_sync(0xffffffffu, in && p.shut[at] >= 0);
      double sum = in && lane < (cuts ? __ffs(cuts) : 32) ? p.sums[at] : 0.0;
      if (next < chunks && !cuts) {
        const float* part = p.adots + (anchor_of(x.a, next) * p.Hv + hv) * p.parts;
        for (int j = lane; j < p.parts; j += 32) sum += static_cast<double>(part[j]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) later[i] = sum, shut[i] = p.shut[hv * p.slots + slot];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < x.n * heads; i += kGateThreads) {
      float* at = dg + static_cast<int64_t>(i / heads) * p.Hv + first + i % heads;
      if (i / heads > shut[i % heads]) *at = static_cast<float>(later[i % heads] + static_cast<double>(*at));
    }
    __syncthreads();
  }
}

int launch_delta_gates(const DeltaCall& c, cudaStream_t stream) {
  const int64_t slots = delta_slots(c.s.total, c.s.nseq);
  const GateArgs a{c.cu, c.sums, c.shut, c.adots, c.dg, c.s.total, c.s.nseq, c.s.Hv, delta_tiles(c.s.V) * kRowWarps, slots};
  return launch_pdl(cattn_delta_gates_kernel, dim3(static_cast<unsigned>(slots)), dim3(kGateThreads), 0, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_delta_grads(const DeltaCall& c, cudaStream_t stream) {
  GradArgs a{};
  int rc = bind_context(), sms = 0;
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mo, c.d_o, c.s.total, c.s.Hv, c.s.V, kDelta, kColumns);
  if (rc == CCONV_OK)
    rc = encode_tile_map(&a.mv, Rows{c.dv, int64_t(c.s.Hv) * c.s.V, c.s.V}, c.s.total, c.s.Hv, c.s.V, kDelta, kColumns);
  if (rc == CCONV_OK) rc = sm_count(&sms);
  if (rc != CCONV_OK) return rc;
  a.g = c.g;
  a.cu = c.cu;
  a.u = c.u, a.heads = c.heads, a.ends = c.ends, a.rest = c.rest;
  a.odots = c.odots, a.vdots = c.vdots, a.bdots = c.bdots;
  a.dq = c.dq, a.dk = c.dk, a.dg = c.dg, a.dbeta = c.dbeta;
  a.sums = c.sums, a.shut = c.shut;
  a.scale = c.scale;
  a.total = c.s.total, a.nseq = c.s.nseq, a.Hk = c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.tiles = delta_tiles(c.s.V);
  a.fresh = c.initial == nullptr;
  a.items = delta_slots(c.s.total, c.s.nseq) * c.s.Hk;
  const int64_t ctas = a.items < sms ? a.items : sms;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_delta_grads_kernel), kGradBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(cattn_delta_grads_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kGradThreads), kGradBytes,
                    stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cattn
