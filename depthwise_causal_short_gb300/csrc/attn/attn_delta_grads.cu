// attn_delta_grads.cu -- the gated delta rule's dq and dk, and the sums that give dg and dbeta.
//
// With S_0 and D, the state before a chunk and the gradient of the state behind it, known (the chains
// left their first bf16 terms), all chunks are done at once; per chunk and value head
//   X = scale (do u^T) . L (s <= t),   Y = (dv u^T) . L (s < t)
//   dq = X K                        + scale ef . (do S_0^T)
//   dk = X^T Q - (Y + Y^T) K + eb . (u D^T) - ef . (dv S_0^T)
// summed over the value heads of a key head in the CTA's registers.  do and dv lie one over the other
// as a first operand of 128 rows, and so do dq and dk as results:
//   [do; dv] u^T       (u in two terms)      -> X, -Y as bf16
//   [do; dv] S_0^T     rows scaled by scale ef and -ef afterwards
//   [  ; u ] D^T       rows 64.. scaled by eb afterwards
//   [X; -Y] K,  [0; -Y^T] K,  [0; X^T] Q
// A CTA goes through (chunk, key head) items; do, dv and the tiles of S_0 and D come by TMA, 64 columns
// of V at a time, u is made from z.  Roundings to bf16: X, Y, S_0, D and u (for D), once each, and dv,
// which is an output.
//
// dg_t is the sum of o_i . do_i - v_i . dv_i over the tokens i >= t of the sequence.
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
constexpr int kStepOut = 2 * kHalf;                       // do over dv
constexpr int kStepState = 2 * kStatePanel;               // two tiles of S_0; of D
constexpr int kStepU = 2 * kHalf;                         // second terms of u over the first ones
constexpr int kStepBytes = kStepOut + 2 * kStepState + kStepU;
constexpr int kGradStages = 2;
constexpr int kOffGradKq = kGradStages * kStepBytes;
constexpr int kOffZero = kOffGradKq + kStageKq;           // zeros, X, -Y: 64 rows each
constexpr int kOffXy = kOffZero + kHalf;
constexpr int kOffLogs = kOffXy + 2 * kHalf;              // log2 decays, and their sums from token 32 on
constexpr int kOffGradBars = kOffLogs + 4 * kDelta * 4;
constexpr int kGradBytes = kOffGradBars + 20 * 8 + 1024;
static_assert(kGradBytes <= 232448, "shared memory of one CTA");
// columns of TMEM
constexpr int kAccXy = 0, kAccState = 64, kAccEnd = 192, kAccIntra = 320;

struct GradArgs {
  CUtensorMap mq, mk, mo, mv;  // q, k, do, dv
  Gates g, beta;
  const int32_t* cu;
  const float* z;
  const uint8_t *heads, *ends;
  uint16_t *dq, *dk;
  float scale;
  int total, nseq, Hk, Hv, K, V, tiles;
  int64_t items;  // slots * Hk
};

__global__ void __launch_bounds__(kChainThreads, 1) cattn_delta_grads_kernel(const __grid_constant__ GradArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem = smem_addr(base);
  const uint32_t full = smem + kOffGradBars, empty = full + 8 * kGradStages;      // tiles of a step
  const uint32_t uready = empty + 8 * kGradStages;                                // u of a step
  const uint32_t kqfull = uready + 8 * kGradStages, kqempty = kqfull + 8;         // an item's K and Q
  const uint32_t xyfull = kqempty + 8, xyready = xyfull + 8;                      // a head's X and Y
  const uint32_t headfull = xyready + 8, headfree = headfull + 8;                 // a head's sums
  const uint32_t gready = headfree + 8, alldone = gready + 8;                      // a head's gates
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ratio = p.Hv / p.Hk, steps = (p.V + 63) / 64;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kGradStages; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
      bar_init(uready + 8 * i, kRowWarps);
    }
    bar_init(kqfull, 1);
    bar_init(kqempty, 1);
    bar_init(xyfull, 1);
    bar_init(xyready, kRowWarps);
    bar_init(headfull, 1);
    bar_init(headfree, kRowWarps);
    bar_init(gready, 1);
    bar_init(alldone, 1);
    cconv::fence_mbar_init();
  }
  for (int i = threadIdx.x; i < kHalf / 16; i += kChainThreads) sts128(smem + kOffZero + i * 16, 0, 0, 0, 0);
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
    int step = 0, item = 0, part = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      const int hk = static_cast<int>(at % p.Hk);
      const int64_t slot = at / p.Hk;
      int row0, n;
      if (!find_chunk(p.cu, p.nseq, p.total, slot, lane, row0, n)) continue;
      if (elect_one()) {
        const int panels = p.K > kPanelCols ? 2 : 1;
        if (item > 0) ok = DELTA_WAIT(kqempty, item - 1);
        if (ok) {
          bar_expect(kqfull, panels * 2 * kSideBytes);
          for (int j = 0; j < panels; ++j) {
            load_box(smem + kOffGradKq + j * kPanelBytes, &p.mk, kqfull, j * kPanelCols, hk, row0);
            load_box(smem + kOffGradKq + j * kPanelBytes + kSideBytes, &p.mq, kqfull, j * kPanelCols, hk, row0);
          }
          part = 1;
        }
        for (int h = 0; h < ratio && ok; ++h) {
          const int hv = hk * ratio + h;
          for (int s = 0; s < steps && ok; ++s, ++step) {
            const int st = step % kGradStages;
            if (step >= kGradStages && !(ok = DELTA_WAIT(empty + 8 * st, step / kGradStages - 1))) break;
            const int tiles = min(2, p.tiles - 2 * s);
            const uint32_t dst = smem + st * kStepBytes, bar = full + 8 * st;
            bar_expect(bar, kStepOut + 2 * tiles * kStatePanel);
            load_box(dst, &p.mo, bar, s * 64, hv, row0);
            load_box(dst + kHalf, &p.mv, bar, s * 64, hv, row0);
            const int64_t from = ((slot * p.Hv + hv) * p.tiles + 2 * s) * kStatePanel;
            bulk_load(dst + kStepOut, p.heads + from, tiles * kStatePanel, bar);
            bulk_load(dst + kStepOut + kStepState, p.ends + from, tiles * kStatePanel, bar);
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
      step = __reduce_max_sync(0xffffffffu, step);
      if (ok) ++item, part = 0;
    }
    item += __any_sync(0xffffffffu, part);
    if (elect_one()) {
      drain(kqfull, item);
      for (int st = 0; st < kGradStages; ++st) drain(full + 8 * st, (step - st + kGradStages - 1) / kGradStages);
    }
  } else if (warp == 1) {
    // ---- products ----
    int step = 0, item = 0, head = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      int row0, n;
      if (!find_chunk(p.cu, p.nseq, p.total, at / p.Hk, lane, row0, n)) continue;
      if (elect_one()) {
        const int width = p.K > kPanelCols ? 128 : 64;  // channels of the results
        const uint32_t d_xy = mma_desc(kDelta, false, false), d_state = mma_desc(width, false, false);
        const uint32_t d_rows = mma_desc(width, false, true), d_cols = mma_desc(width, true, true);
        ok = DELTA_WAIT(kqfull, item);
        for (int h = 0; h < ratio && ok; ++h, ++head) {
          if (head > 0 && !(ok = DELTA_WAIT(headfree, head - 1))) break;
          tc_fence_after();
          for (int s = 0; s < steps && ok; ++s, ++step) {
            const int st = step % kGradStages;
            const uint32_t src = smem + st * kStepBytes, u = src + kStepOut + 2 * kStepState;
            const int ks = (min(64, p.V - 64 * s) + 15) / 16;
            if (!(ok = DELTA_WAIT(full + 8 * st, step / kGradStages))) break;
            if (!(ok = DELTA_WAIT(uready + 8 * st, step / kGradStages))) break;
            tc_fence_after();
            const uint64_t a = tile_desc(src, 0), lo = tile_desc(u, 0), hi = tile_desc(u + kHalf, 0);
#pragma unroll 1
            for (int j = 0; j < ks; ++j) {
              mma_ss(tmem + kAccXy, a + 2 * j, hi + 2 * j, d_xy, s + j > 0);
              mma_ss(tmem + kAccXy, a + 2 * j, lo + 2 * j, d_xy, true);
            }
            if (s + 1 == steps) mma_commit(xyfull);
#pragma unroll 1
            for (int j = 0; j < ks; ++j) {
              const uint64_t state = term_desc(src + kStepOut + (j >> 1) * kStatePanel, 0) + 2 * (j & 1);
              const uint64_t end = term_desc(src + kStepOut + kStepState + (j >> 1) * kStatePanel, 0) + 2 * (j & 1);
              mma_ss(tmem + kAccState, a + 2 * j, state, d_state, s + j > 0);
              mma_ss(tmem + kAccEnd, lo + 2 * j, end, d_state, s + j > 0);
            }
            mma_commit(empty + 8 * st);
          }
          if (!ok || !(ok = DELTA_WAIT(xyready, head))) break;
          tc_fence_after();
          const uint64_t k = tile_desc(smem + kOffGradKq, kPanelBytes);
          const uint64_t q = tile_desc(smem + kOffGradKq + kSideBytes, kPanelBytes);
          const uint64_t xy = tile_desc(smem + kOffXy, 0);
          const uint64_t xt = tile_desc(smem + kOffZero, kHalf), yt = tile_desc(smem + kOffZero, 2 * kHalf);
#pragma unroll 1
          for (int j = 0; j < kDelta / 16; ++j) {
            mma_ss(tmem + kAccIntra, xy + 2 * j, k + j * kRowStep, d_rows, h + j > 0);
            mma_ss(tmem + kAccIntra, yt + j * kRowStep, k + j * kRowStep, d_cols, true);
            mma_ss(tmem + kAccIntra, xt + j * kRowStep, q + j * kRowStep, d_cols, true);
          }
          mma_commit(headfull);
        }
        if (ok) mma_commit(kqempty);
      }
      ok = __all_sync(0xffffffffu, ok);
      step = __reduce_max_sync(0xffffffffu, step);
      head = __reduce_max_sync(0xffffffffu, head);
      ++item;
    }
    if (elect_one()) {
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (warp >= 4) {
    // ---- rows ----
    const int quarter = warp % 4, cg = warp / 4 - 1;
    const int row = quarter * 32 + lane, t = row & (kDelta - 1);
    const bool dq = quarter < 2;                      // this thread's row is one of dq; or of dk
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const int piece = (quarter >> 1) * 2 + cg;        // 16 columns of u of token t
    const int tid = threadIdx.x - 128;
    float* logs = reinterpret_cast<float*>(base + kOffLogs);
    int step = 0, item = 0, head = 0;
    for (int64_t at = blockIdx.x; at < p.items && ok; at += gridDim.x) {
      const int hk = static_cast<int>(at % p.Hk);
      int row0, n;
      if (!find_chunk(p.cu, p.nseq, p.total, at / p.Hk, lane, row0, n)) continue;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      for (int h = 0; h < ratio && ok; ++h, ++head) {
        const int hv = hk * ratio + h;
        // gates: [0, 64) log2 decays, [64, 128) their sums from token 0 or 32 on, [128, 192) ef, [192, 256) eb
        if (warp == 4) {
          if (head > 0 && !(ok = DELTA_WARP_WAIT(headfree, head - 1))) break;  // the last head's are read
          float g[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) g[j] = 2 * lane + j < n ? kLog2e * p.g.at(row0 + 2 * lane + j, hv) : 0.f;
          float up = g[0] + g[1], down = up, half = up;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, up, o), y = __shfl_down_sync(0xffffffffu, down, o);
            if (lane >= o) up += x;
            if (lane + o < 32) down += y;
          }
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, half, o, 16);
            if ((lane & 15) >= o) half += x;
          }
          float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
          float start = __shfl_up_sync(0xffffffffu, half, 1, 16);
          if (lane == 0) before = 0.f;
          if (lane == 31) after = 0.f;
          if ((lane & 15) == 0) start = 0.f;
          const int i = 2 * lane;
          logs[i] = g[0], logs[i + 1] = g[1];
          logs[64 + i] = start + g[0], logs[64 + i + 1] = start + g[0] + g[1];
          logs[128 + i] = exp2_fast(before + g[0]), logs[128 + i + 1] = exp2_fast(before + g[0] + g[1]);
          logs[192 + i] = exp2_fast(g[1] + after), logs[192 + i + 1] = exp2_fast(after);
          __syncwarp();
          if (lane == 0) bar_arrive(gready);
        }
        if (!(ok = DELTA_WARP_WAIT(gready, head))) break;
        const float beta = t < n ? __ldg(p.beta.p + (row0 + t) * p.beta.st + hv * p.beta.sh) : 0.f;
        for (int s = 0; s < steps; ++s, ++step) {
          // u of token t, 16 columns, in two terms
          const int st = step % kGradStages, col = s * 64 + piece * 16;
          float4 z[4];
          const float4* src = reinterpret_cast<const float4*>(p.z + (static_cast<int64_t>(row0 + t) * p.Hv + hv) * p.V + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < n && col + 4 * i < p.V) z[i] = src[i];
          }
          if (step >= kGradStages && !(ok = DELTA_WARP_WAIT(empty + 8 * st, step / kGradStages - 1))) break;
          const uint32_t u = smem + st * kStepBytes + kStepOut + 2 * kStepState;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x[8] = {beta * z[2 * i].x, beta * z[2 * i].y, beta * z[2 * i].z, beta * z[2 * i].w,
                                beta * z[2 * i + 1].x, beta * z[2 * i + 1].y, beta * z[2 * i + 1].z, beta * z[2 * i + 1].w};
            uint4 w[kTerms];
            split8(x, w);
            const uint32_t to = u + swizzled(t, piece * 2 + i);
            sts128(to + kHalf, w[0].x, w[0].y, w[0].z, w[0].w);
            sts128(to, w[1].x, w[1].y, w[1].z, w[1].w);
          }
          cconv::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive(uready + 8 * st);
        }
        if (!ok) break;
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
        if (!(ok = DELTA_WARP_WAIT(xyfull, head))) break;
        tc_fence_after();
        {
          uint32_t x[32];
          tmem_ld32(tmem + lanes + kAccXy + cg * 32, x);
          tmem_wait_ld();
          tmem_use32(x);
          const float f = dq ? p.scale : -1.f;
          float e = cg == 0 && t >= 32 ? logs[64 + t] : 0.f;
#pragma unroll
          for (int i = 31; i >= 0; --i) {
            const int s = cg * 32 + i;
            if (i < 31 && s < t) e += logs[s + 1];
            if (i == 31 && cg == 1 && s < t) e += logs[s + 1 < kDelta ? s + 1 : s];
            const float v = f * __uint_as_float(x[i]) * exp2_fast(e);
            x[i] = __float_as_uint(t < n && (s < t || (dq && s == t)) ? v : 0.f);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = f2_to_bf16x2(pair(x, 4 * i + j));
            sts128(smem + kOffXy + swizzled(row, cg * 4 + i), w[0], w[1], w[2], w[3]);
          }
        }
        cconv::fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(xyready);
        if (!(ok = DELTA_WARP_WAIT(headfull, head))) break;
        tc_fence_after();
        const float ef = logs[128 + t], eb = logs[192 + t], f = dq ? p.scale * ef : -ef;
        const bool last = h + 1 == ratio;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int c = cg * 64 + b * 16;
          if (c >= p.K) continue;
          uint32_t x[16], y[16], w[16];
          tmem_ld16(tmem + lanes + kAccState + c, x);
          tmem_ld16(tmem + lanes + kAccEnd + c, y);
          if (last) tmem_ld16(tmem + lanes + kAccIntra + c, w);
          tmem_wait_ld();
          tmem_use16(x);
          tmem_use16(y);
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
        uint16_t* dst = (dq ? p.dq : p.dk) + (static_cast<int64_t>(row0 + t) * p.Hk + hk) * p.K + cg * 64;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = f2_to_bf16x2(f2_pack(acc[8 * i + 2 * j], acc[8 * i + 2 * j + 1]));
          if (cg * 64 + 8 * i < p.K) *reinterpret_cast<uint4*>(dst + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
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

// dg and dbeta of one sequence and value head by one CTA, from the last token on, kGateThreads tokens
// at a time.  The running sum is kept in 64 bits: it adds up terms of both signs over the whole
// sequence, and what is left of them is small where a head forgets fast.
constexpr int kGateThreads = 256;
struct GateArgs {
  const int32_t* cu;
  const float *odots, *vdots, *bdots;
  float *dg, *dbeta;
  int total, Hv, parts;
};
__global__ void __launch_bounds__(kGateThreads) cattn_delta_gates_kernel(const GateArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ double sums[2][kGateThreads / 32];
  const int hv = static_cast<int>(blockIdx.x % p.Hv), seq = static_cast<int>(blockIdx.x / p.Hv);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int a, b;
  sequence_rows(p.cu, seq, p.total, a, b);
  if (p.cu[seq] < 0 || p.cu[seq + 1] < p.cu[seq] || p.cu[seq + 1] > p.total) return;
  double carry = 0.0;
  int turn = 0;
  for (int64_t top = b; top > a; top -= kGateThreads, turn ^= 1) {
    const int64_t t = top - 1 - threadIdx.x;
    double x = 0.0;
    if (t >= a) {
      float db = 0.f;
      for (int i = 0; i < p.parts; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * p.Hv + hv) * p.total + t;
        x += static_cast<double>(p.odots[at]) - static_cast<double>(p.vdots[at]);
        db += p.bdots[at];
      }
      p.dbeta[t * p.Hv + hv] = db;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[turn][warp] = x;
    __syncthreads();
    double before = carry;
#pragma unroll
    for (int i = 0; i < kGateThreads / 32; ++i) {
      if (i < warp) before += sums[turn][i];
      carry += sums[turn][i];
    }
    if (t >= a) p.dg[t * p.Hv + hv] = static_cast<float>(before + x);
  }
}

int launch_delta_gates(const DeltaCall& c, cudaStream_t stream) {
  GateArgs a{c.cu, c.odots, c.vdots, c.bdots, c.dg, c.dbeta, c.s.total, c.s.Hv, 2 * delta_tiles(c.s.V)};
  const int64_t ctas = static_cast<int64_t>(c.s.nseq) * c.s.Hv;
  return launch_pdl(cattn_delta_gates_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kGateThreads), 0, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_delta_grads(const DeltaCall& c, cudaStream_t stream) {
  GradArgs a{};
  int rc = bind_context(), sms = 0;
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K, kDelta);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mo, c.d_o, c.s.total, c.s.Hv, c.s.V, kDelta);
  if (rc == CCONV_OK)
    rc = encode_tile_map(&a.mv, Rows{c.dv, int64_t(c.s.Hv) * c.s.V, c.s.V}, c.s.total, c.s.Hv, c.s.V, kDelta);
  if (rc == CCONV_OK) rc = sm_count(&sms);
  if (rc != CCONV_OK) return rc;
  a.g = c.g, a.beta = c.beta;
  a.cu = c.cu;
  a.z = c.z, a.heads = c.heads, a.ends = c.ends;
  a.dq = c.dq, a.dk = c.dk;
  a.scale = c.scale;
  a.total = c.s.total, a.nseq = c.s.nseq, a.Hk = c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.tiles = delta_tiles(c.s.V);
  a.items = delta_slots(c.s.total, c.s.nseq) * c.s.Hk;
  const int64_t ctas = a.items < sms ? a.items : sms;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_delta_grads_kernel), kGradBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(cattn_delta_grads_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kChainThreads), kGradBytes,
                    stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cattn
