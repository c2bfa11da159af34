// attn_chunk_bwd.cu -- the gradient of the chunked linear attention on the tensor cores.
//
// Two sweeps over the same ranges of units as the forward (attn_chunk.cuh); rows of a unit's
// [128, 128] score tiles are its lanes:
//
//   KV = false, first chunk to last, rows t (queries):
//     M1 = dO V^T, M2 = Q K^T, P = M1 . L
//     dq = scale (P K + er . (dO S^T)),   S <- total S + (kw . K)^T V
//   KV = true, last chunk to first, rows s (keys):
//     M1 = V dO^T, M2 = K Q^T, P1 = M1 . L^T, P2 = M2 . L^T
//     dk = scale (P1 Q + kw . (V D^T)),   dv = scale (P2 dO + kw . (K D))
//     D <- total D + (er . Q)^T dO
//
// For dg (see attn_linear.cu) every unit also writes, in fp32, the sums over its rows of the
// pairs that are not a token with itself: inside the chunk scale * sum M1 . M2 . L without the
// diagonal, whose factors come from fp32 products of the inputs and are never rounded; across
// chunks scale * er * q . (dO S^T) and scale * kw * k . (V D^T), for which S and D are read as
// two bf16 terms (16 bits).
//
// Roles of the 16 warps are the forward's: tiles, matrix products, gates; four warps turn the
// score tiles into P, eight keep the state and finish the outputs.  The ring's four slots hold
// one tile each of v, do, k and q, refilled as soon as its last reader is done.  TMEM:
//   KV = false  [0,128) M1, then P   [128,256) M2, then P K   [256,384) dO S^T   [384,512) K^T V
//   KV = true   [0,128) M1, then P1 | Q^T dO (columns 0-63)   [128,256) M2, then P2 | Q^T dO (64-)
//               [256,384) dk         [384,512) dv: V D^T and K D are scaled in place, P Q and
//               P dO accumulate on them
#include "attn_chunk.cuh"
#include "attn_chunk_host.h"

namespace cattn {

static __device__ unsigned g_fault_bwd;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_bwd, sizeof(*out))) !=
          cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_bwd, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

constexpr int kStateWarps = 8;
constexpr int kBwdThreads = 512;
constexpr int kBwdGates = 2;
constexpr int kBlock = 16;                        // tokens of one decayed block
constexpr int kBlockPanel = kBlock * 128;
constexpr int kBlockTile = 2 * kBlockPanel;
constexpr int kBlockBytes = kSplit * kBlockTile;
enum Slot : int { kV = 0, kDo = 1, kK = 2, kQ = 3, kBwdSlots = 4 };

// shared memory, from a 1024-byte boundary
constexpr int kOffKp = kBwdSlots * kTileBytes;          // two blocks of decayed rows
constexpr int kOffS = kOffKp + 2 * kBlockBytes;         // the state as two bf16 terms
constexpr int kOffGates = kOffS + 2 * kTileBytes;
constexpr int kOffBars = kOffGates + kBwdGates * sizeof(Gate);
constexpr int kBwdBytes = kOffBars + 40 * 8 + 1024;
static_assert(kBwdBytes <= 232448, "shared memory of one CTA");

struct BwdArgs {
  CUtensorMap mq, mk, mv, mo;
  Plan plan;
  Gates g;
  Slots slots;
  const float* initial;
  float* dinit;             // KV: [nseq, Hv, K, V] or NULL
  uint16_t *dq, *dk, *dv;   // dq or dk in bf16 where one unit makes a row of them, else
  float* part;              // [units' (head, tile)][total][K] partial sums
  float* dots;              // [3][heads * tiles][total]
  const float* carry;       // states handed on
  const float* decay;
  float scale;
  int rows, ratio, Hk, Hv, K, V;
  int wide_k, wide_v;       // rows of dq, dk and of dv allow 32-byte stores
};

#define CATTN_WAIT(bar, parity) \
  (wait_phase((bar), static_cast<uint32_t>(parity) & 1u, gave_up, &g_fault_bwd))
#define CATTN_WARP_WAIT(bar, parity) (__all_sync(0xffffffffu, CATTN_WAIT(bar, parity)))

// Stores 32 fp32 values times `f` as bf16 to columns [c, c + 32) of a row of `width` columns.
__device__ __forceinline__ void store_bf16(uint16_t* row, int c, int width, bool wide,
                                           const uint32_t* x, float f) {
  uint32_t y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    y[i] = pack_bf16(f * __uint_as_float(x[2 * i]), f * __uint_as_float(x[2 * i + 1]));
  if (wide && c + 32 <= width) {
    stg256(row + c, y);
    stg256(row + c + 16, y + 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 8 * i < width)
        *reinterpret_cast<uint4*>(row + c + 8 * i) =
            make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
  }
}

// The same in fp32 (rows of K floats, K % 8 == 0, on 32-byte boundaries).
__device__ __forceinline__ void store_f32(float* row, int c, int width, const uint32_t* x, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __float_as_uint(f * __uint_as_float(x[8 * i + j]));
    if (c + 8 * i < width) stg256(row + c + 8 * i, y);
  }
}

// Dot of 32 fp32 values with columns [c, c + 32) of row `row` of a bf16 tile.
__device__ __forceinline__ float dot_tile(uint32_t tile, int row, int c, const uint32_t* x) {
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = c + 8 * i;
    const uint4 w = lds128_at(tile + (col / kPanelCols) * kPanelBytes +
                              swizzled(row, (col % kPanelCols) / 8));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dot = fmaf(__uint_as_float(u[j] << 16), __uint_as_float(x[8 * i + 2 * j]), dot);
      dot = fmaf(__uint_as_float(u[j] & 0xffff0000u), __uint_as_float(x[8 * i + 2 * j + 1]), dot);
    }
  }
  return dot;
}

template <bool KV>
__global__ void __launch_bounds__(kBwdThreads, 1)
    cattn_linear_chunk_bwd_kernel(const __grid_constant__ BwdArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Gate* gates = reinterpret_cast<Gate*>(base + kOffGates);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + kOffBars);
  uint64_t *full = bars, *empty = bars + kBwdSlots;
  uint64_t *gfull = empty + kBwdSlots, *gempty = gfull + kBwdGates;
  uint64_t *kpfull = gempty + kBwdGates, *kpempty = kpfull + 2;
  uint64_t *fixed = kpempty + 2, *scfull = fixed + 1, *pfull = scfull + 1, *kvfull = pfull + 1;
  uint64_t *kvfree = kvfull + 1, *sfull = kvfree + 1, *sempty = sfull + 1, *infull = sempty + 1;
  uint64_t *scaled = infull + 1, *ofull = scaled + 1, *ofree = ofull + 1, *alldone = ofree + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(alldone + 1);
  volatile int* gave_up = reinterpret_cast<int*>(tmem_at + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBwdSlots; ++i) {
      cconv::mbar_init(&full[i], 1);
      // the tile that the rows' dots read goes when the state warps are done with it
      cconv::mbar_init(&empty[i], i == (KV ? kK : kQ) ? kStateWarps : 1);
    }
    for (int i = 0; i < kBwdGates; ++i) {
      cconv::mbar_init(&gfull[i], 1);
      cconv::mbar_init(&gempty[i], 4 + kStateWarps + 1);
    }
    for (int i = 0; i < 2; ++i) {
      cconv::mbar_init(&kpfull[i], kStateWarps);
      cconv::mbar_init(&kpempty[i], 1);
    }
    cconv::mbar_init(fixed, kStateWarps);
    cconv::mbar_init(scfull, 1);
    cconv::mbar_init(pfull, 4);
    cconv::mbar_init(kvfull, 1);
    cconv::mbar_init(kvfree, kStateWarps);
    cconv::mbar_init(sfull, kStateWarps);
    cconv::mbar_init(sempty, 1);
    cconv::mbar_init(infull, 1);
    cconv::mbar_init(scaled, kStateWarps);
    cconv::mbar_init(ofull, 1);
    cconv::mbar_init(ofree, kStateWarps);
    cconv::mbar_init(alldone, 1);
    *gave_up = 0;
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_at, 512);
  if (warp == 0 && lane == 0) {
    cconv::prefetch_tensormap(&p.mq);
    cconv::prefetch_tensormap(&p.mk);
    cconv::prefetch_tensormap(&p.mv);
    cconv::prefetch_tensormap(&p.mo);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t smem = smem_addr(base);
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();

  int nch;
  const int64_t units = unit_count(p.plan, nch);
  const int64_t parts = min(static_cast<int64_t>(gridDim.x), units);
  Range range{0, 0};
  if (blockIdx.x < parts) range = range_of(units, parts, blockIdx.x);
  const int64_t count = range.u1 - range.u0, start = KV ? range.u1 - 1 : range.u0;
  const int pk = p.K > kPanelCols ? 2 : 1;
  const uint32_t av = smem + kV * kTileBytes, ao = smem + kDo * kTileBytes;
  const uint32_t ak = smem + kK * kTileBytes, aq = smem + kQ * kTileBytes;

  if (count > 0) {
  if (warp == 0) {
    // ---- tiles ----
    if (lane == 0) {
      Walker w;
      w.seek(&p.plan, nch, start);
      int use = 0;
      bool ok = true;
      for (int64_t i = 0; i < count && ok; ++i) {
        if (w.rows() > 0) {
          const int hv = w.ht / p.plan.tiles, vt = w.ht % p.plan.tiles;
          const int hk = hv / p.ratio, row = w.row0();
          const int pv = p.V - vt * 128 > kPanelCols ? 2 : 1;
          for (int j = 0; j < kBwdSlots; ++j) {
            if (use > 0 && !(ok = CATTN_WAIT(&empty[j], use - 1))) break;
            const bool isv = j == kV || j == kDo;
            const CUtensorMap* map = j == kV ? &p.mv : j == kDo ? &p.mo : j == kK ? &p.mk : &p.mq;
            const int panels = isv ? pv : pk;
            cconv::mbar_arrive_expect_tx(&full[j], panels * kPanelBytes);
            for (int c = 0; c < panels; ++c)
              cconv::tma_load_3d(base + j * kTileBytes + c * kPanelBytes, map, &full[j],
                                 (isv ? vt * 128 : 0) + c * kPanelCols, isv ? hv : hk, row);
          }
          if (!ok) break;
          ++use;
        }
        if (i + 1 < count) w.step<KV>();
      }
      // one copy into each slot for each use (a use that gave up half-way counts none: its
      // copies are waited for too, as the phase after)
      for (int j = 0; j < kBwdSlots; ++j) {
        if (use > 0) (void)cconv::mbar_wait_bounded(&full[j], (use - 1) & 1, cconv::kDrainLimitNs);
        if (!ok) (void)cconv::mbar_wait_bounded(&full[j], use & 1, cconv::kDrainLimitNs);
      }
    }
  } else if (warp == 1) {
    // ---- matrix products ----
    if (lane == 0) {
      int use = 0, subs = 0, pubs = 0, fixes = 0, kvs = 0;
      bool ok = true;
      const int kk = (p.K + 15) / 16, nk = kk * 16;
      for (int unit = 0; unit < count && ok; ++unit) {
        const int gs = unit % kBwdGates;
        if (!(ok = CATTN_WAIT(&gfull[gs], unit / kBwdGates))) break;
        const Gate& gt = gates[gs];
        const int n = gt.n, flags = gt.flags, ht = gt.ht;
        if (n > 0) {
          const int vw = min(128, p.V - ht % p.plan.tiles * 128);
          const int kv = (vw + 15) / 16, nv = kv * 16;
          const int steps = (n + 15) / 16;
          for (int j = 0; j < kBwdSlots && ok; ++j) ok = CATTN_WAIT(&full[j], use);
          if (!ok) break;
          if (n < kChunk) {
            if (!(ok = CATTN_WAIT(fixed, fixes))) break;
            ++fixes;
          }
          // the score tiles overwrite the last chunk's P, outputs and state product
          if (use > 0) {
            if (!(ok = CATTN_WAIT(ofull, use - 1))) break;
            if (!(ok = CATTN_WAIT(ofree, use - 1))) break;
          }
          if (KV && kvs > 0 && !(ok = CATTN_WAIT(kvfree, kvs - 1))) break;
          tc_fence_after();
          const uint32_t ds = mma_desc(128, false, false);
          for (int j = 0; j < kv; ++j) {
            const uint32_t off = (j / 4) * kPanelBytes + (j % 4) * 32;
            mma_ss(tmem, tile_desc((KV ? av : ao) + off, 0), tile_desc((KV ? ao : av) + off, 0), ds,
                   j > 0);
          }
          for (int j = 0; j < kk; ++j) {
            const uint32_t off = (j / 4) * kPanelBytes + (j % 4) * 32;
            mma_ss(tmem + 128, tile_desc((KV ? ak : aq) + off, 0), tile_desc((KV ? aq : ak) + off, 0),
                   ds, j > 0);
          }
          mma_commit(scfull);
          if (flags & kHasState) {
            if (!(ok = CATTN_WAIT(sfull, pubs))) break;
            ++pubs;
            tc_fence_after();
            // dO S^T or V D^T: the state's rows are the output's columns, its columns are summed
            const uint32_t d = mma_desc(nk, false, false);
            for (int term = 0; term < 2; ++term)
              for (int j = 0; j < kv; ++j) {
                const uint32_t off = (j / 4) * kPanelBytes + (j % 4) * 32;
                mma_ss(tmem + 256, tile_desc((KV ? av : ao) + off, 0),
                       tile_desc(smem + kOffS + term * kTileBytes + off, 0), d, term + j > 0);
              }
            if (KV) {
              const uint32_t dd = mma_desc(nv, false, true);
              for (int j = 0; j < kk; ++j)
                mma_ss(tmem + 384, tile_desc(ak + (j / 4) * kPanelBytes + (j % 4) * 32, 0),
                       tile_desc(smem + kOffS + j * 2048, kPanelBytes), dd, j > 0);
            }
            mma_commit(infull);
            mma_commit(sempty);
          }
          mma_commit(KV ? &empty[kV] : &empty[kDo]);
          if (KV) {
            if (!(ok = CATTN_WAIT(pfull, use))) break;
            tc_fence_after();
          }
          if (flags & kNeedKv) {
            const uint32_t b = KV ? ao : av;
            const int n0 = KV ? min(nv, 64) : nv;
            const uint32_t d0 = mma_desc(n0, true, true), d1 = mma_desc(nv > 64 ? nv - 64 : 16, true, true);
            for (int blk = 0; blk < steps; ++blk, ++subs) {
              if (!(ok = CATTN_WAIT(&kpfull[subs & 1], subs >> 1))) break;
              tc_fence_after();
              for (int s = 0; s < kSplit; ++s) {
                const uint64_t a = tile_desc(smem + kOffKp + (subs & 1) * kBlockBytes + s * kBlockTile,
                                             kBlockPanel);
                mma_ss(tmem + (KV ? 64 : 384), a, tile_desc(b + blk * 2048, kPanelBytes), d0, blk + s > 0);
                if (KV && nv > 64)
                  mma_ss(tmem + 192, a, tile_desc(b + kPanelBytes + blk * 2048, kPanelBytes), d1,
                         blk + s > 0);
              }
              mma_commit(&kpempty[subs & 1]);
            }
            if (!ok) break;
            mma_commit(kvfull);
            ++kvs;
          }
          if (!KV) {
            mma_commit(&empty[kV]);
            if (!(ok = CATTN_WAIT(pfull, use))) break;
            tc_fence_after();
            const uint32_t d = mma_desc(nk, false, true);
            for (int j = 0; j < steps; ++j)
              mma_ts(tmem + 128, tmem + j * 8, tile_desc(ak + j * 2048, kPanelBytes), d, j > 0);
            mma_commit(ofull);
            mma_commit(&empty[kK]);
          } else {
            const bool add = flags & kHasState;
            if (add) {
              if (!(ok = CATTN_WAIT(scaled, pubs - 1))) break;
              tc_fence_after();
            }
            const uint32_t dk = mma_desc(nk, false, true), dv = mma_desc(nv, false, true);
            for (int j = 0; j < steps; ++j)
              mma_ts(tmem + 256, tmem + j * 8, tile_desc(aq + j * 2048, kPanelBytes), dk, add || j > 0);
            for (int j = 0; j < steps; ++j)
              mma_ts(tmem + 384, tmem + 128 + j * 8, tile_desc(ao + j * 2048, kPanelBytes), dv,
                     add || j > 0);
            mma_commit(ofull);
            mma_commit(&empty[kQ]);
            mma_commit(&empty[kDo]);
          }
          ++use;
        }
        cconv::mbar_arrive(&gempty[gs]);
      }
      mma_commit(alldone);
      (void)cconv::mbar_wait_bounded(alldone, 0, cconv::kDrainLimitNs);
    }
  } else if (warp == 2) {
    // ---- gates ----
    Walker w;
    w.seek(&p.plan, nch, start);
    for (int64_t i = 0; i < count; ++i) {
      const int unit = static_cast<int>(i);
      const int gs = unit % kBwdGates, n = w.rows(), row0 = w.row0();
      const int hv = w.ht / p.plan.tiles;
      float g[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        g[b] = 32 * b + lane < n ? kLog2e * p.g.at(row0 + 32 * b + lane, hv) : 0.f;
      if (unit >= kBwdGates && !CATTN_WARP_WAIT(&gempty[gs], unit / kBwdGates - 1)) break;
      Gate& gt = gates[gs];
      make_gate(gt, g, lane);
      if (lane == 0) {
        gt.row0 = row0;
        gt.n = n;
        gt.ht = w.ht;
        gt.seq = w.seq;
        int f = 0;
        const bool first = KV ? w.last() : w.first(), last = KV ? w.first() : w.last();
        if (i == 0 || first) f |= kSegment;
        if ((f & kSegment) && !first) f |= kMiddle;
        if (!first || (!KV && p.initial)) f |= kHasState;
        if (KV && last && p.dinit) f |= kFinish;
        if ((!last && i + 1 < count) || (f & kFinish)) f |= kNeedKv;
        gt.flags = f;
      }
      __syncwarp();
      if (lane == 0) cconv::mbar_arrive(&gfull[gs]);
      if (i + 1 < count) w.step<KV>();
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- score tiles to P ----
    const int wq = warp - 4, row = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    int use = 0;
    for (int unit = 0; unit < count; ++unit) {
      const int gs = unit % kBwdGates;
      if (!CATTN_WARP_WAIT(&gfull[gs], unit / kBwdGates)) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, row0 = gt.row0, ht = gt.ht;
      if (n > 0) {
        const float own = KV ? gt.ws[row] : gt.lp[row];
        if (!CATTN_WARP_WAIT(scfull, use)) break;
        tc_fence_after();
        float sum = 0.f;  // pairs of different tokens
        for (int b = 0; b < 4; ++b) {
          uint32_t x[32], z[32], y[16], y2[16];
          const bool live = KV ? b >= wq : b <= wq;
          if (live) {
            tmem_ld32(tmem + lanes + b * 32, x);
            tmem_ld32(tmem + lanes + 128 + b * 32, z);
            tmem_wait_ld();
            tmem_use32(x);
            tmem_use32(z);
          }
          if (live && b != wq) {
            float e = KV ? 0.f : own;
            const int lo = KV ? wq + 1 : b + 1, hi = KV ? b : wq;
            for (int i = lo; i < hi; ++i) e += gt.block[i];
            const float ut = KV ? own * exp2_fast(e) : exp2_fast(e);
            const float* cols = (KV ? gt.pe : gt.ws) + b * 32;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 w = *reinterpret_cast<const float2*>(cols + 2 * i);
              const float w0 = ut * w.x, w1 = ut * w.y;
              const float p0 = __uint_as_float(x[2 * i]) * w0, p1 = __uint_as_float(x[2 * i + 1]) * w1;
              const float z0 = __uint_as_float(z[2 * i]), z1 = __uint_as_float(z[2 * i + 1]);
              y[i] = pack_bf16(p0, p1);
              if (KV) y2[i] = pack_bf16(z0 * w0, z1 * w1);
              sum = fmaf(p0, z0, sum);
              sum = fmaf(p1, z1, sum);
            }
          } else if (b == wq) {
            // the diagonal block: the decay as a running product away from the row's token
            float w = 1.f, held = 0.f, held2 = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int c = KV ? i : 31 - i;
              const bool off = KV ? c > lane : c < lane;
              if (off) w *= gt.a[b * 32 + (KV ? c : c + 1)];
              const bool on = off || c == lane;
              const float v = on ? __uint_as_float(x[c]) * w : 0.f;
              const float v2 = on ? __uint_as_float(z[c]) * w : 0.f;
              if (off) sum = fmaf(v, __uint_as_float(z[c]), sum);
              if (i & 1) {
                y[c / 2] = KV ? pack_bf16(held, v) : pack_bf16(v, held);
                if (KV) y2[c / 2] = pack_bf16(held2, v2);
              } else {
                held = v;
                held2 = v2;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = y2[i] = 0;
          }
          // (P's columns [16 b, 16 b + 16) lie in score columns that are read or not needed)
          tmem_st16(tmem + lanes + b * 16, y);
          if (KV) tmem_st16(tmem + lanes + 128 + b * 16, y2);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cconv::mbar_arrive(pfull);
        if (row < n)
          p.dots[static_cast<int64_t>(ht) * p.rows + row0 + row] = p.scale * sum;
        ++use;
      }
      __syncwarp();
      if (lane == 0) cconv::mbar_arrive(&gempty[gs]);
    }
  } else if (warp >= 8) {
    // ---- the state, and the outputs ----
    const int st = threadIdx.x - 256;
    const int half = st / 128, krow = st % 128;  // columns [64 half, 64 half + 64) of row krow
    const uint32_t lanes = static_cast<uint32_t>(krow & ~31) << 16;
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    int use = 0, subs = 0, pubs = 0, kvs = 0;
    bool ok = true;
    for (int unit = 0; unit < count && ok; ++unit) {
      const int gs = unit % kBwdGates;
      if (!(ok = CATTN_WARP_WAIT(&gfull[gs], unit / kBwdGates))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, flags = gt.flags, ht = gt.ht, row0 = gt.row0;
      const int hv = ht / p.plan.tiles, vt = ht % p.plan.tiles;
      const int vw = min(128, p.V - vt * 128);
      const bool has = flags & kHasState;
      if (flags & kSegment) {
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0.f;
        if (flags & kMiddle) {
          // what the ranges before this one (after it, for KV) hand on
          float coef = 1.f;
          const int64_t by = KV ? 1 : -1;
          for (int64_t j = blockIdx.x + by; j >= 0 && j < parts; j += by) {
            const float4* src = reinterpret_cast<const float4*>(p.carry + j * kStateFloats);
            const float d = p.decay[j];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 x = src[(half * 16 + i) * 128 + krow];
              S[4 * i] = fmaf(coef, x.x, S[4 * i]);
              S[4 * i + 1] = fmaf(coef, x.y, S[4 * i + 1]);
              S[4 * i + 2] = fmaf(coef, x.z, S[4 * i + 2]);
              S[4 * i + 3] = fmaf(coef, x.w, S[4 * i + 3]);
            }
            if (d < 0.f) break;
            coef *= d;
            if (coef == 0.f) break;
          }
        } else if (!KV && p.initial && krow < p.K) {
          const int64_t slot = p.slots.of(gt.seq);
          const float* src = p.initial + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128 + half * 64;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (slot >= 0 && half * 64 + 4 * i < vw) x = *reinterpret_cast<const float4*>(src + 4 * i);
            S[4 * i] = x.x, S[4 * i + 1] = x.y, S[4 * i + 2] = x.z, S[4 * i + 3] = x.w;
          }
        }
      }
      if (n > 0) {
        if (n < kChunk) {
          // the tiles whose rows are summed over
          const uint32_t t0 = KV ? aq : ak, t1 = KV ? ao : av;
          if (!(ok = CATTN_WARP_WAIT(&full[KV ? kQ : kK], use))) break;
          zero_rows(t0, pk, n, st, kStateWarps * 32);
          if (!(ok = CATTN_WARP_WAIT(&full[KV ? kDo : kV], use))) break;
          zero_rows(t1, vw > kPanelCols ? 2 : 1, n, st, kStateWarps * 32);
          cconv::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) cconv::mbar_arrive(fixed);
        }
        if (has) {
          if (pubs > 0 && !(ok = CATTN_WARP_WAIT(sempty, pubs - 1))) break;
          ++pubs;
          const uint32_t dst = smem + kOffS + half * kPanelBytes;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = S[8 * i + 2 * j], b = S[8 * i + 2 * j + 1];
              hi[j] = pack_bf16(a, b);
              lo[j] = pack_bf16(a - __uint_as_float(hi[j] << 16),
                                b - __uint_as_float(hi[j] & 0xffff0000u));
            }
            sts128(dst + swizzled(krow, i), hi[0], hi[1], hi[2], hi[3]);
            sts128(dst + kTileBytes + swizzled(krow, i), lo[0], lo[1], lo[2], lo[3]);
          }
          cconv::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) cconv::mbar_arrive(sfull);
        }
        const int steps = (n + 15) / 16;
        if (flags & kNeedKv) {
          if (!(ok = CATTN_WARP_WAIT(&full[KV ? kQ : kK], use))) break;
          const uint32_t src = KV ? aq : ak;
          const int r = st / 16, piece = st % 16;  // one 16-byte piece of one token
          for (int b = 0; b < steps; ++b, ++subs) {
            if (subs >= 2 && !(ok = CATTN_WARP_WAIT(&kpempty[subs & 1], (subs >> 1) - 1))) break;
            const int t = b * kBlock + r;
            const float w = KV ? gt.er[t] : gt.kw[t];
            if (piece < 8 * pk) {
              const int q = piece / 8, at8 = piece % 8;
              uint32_t hi[4], mid[4], lo[4];
              const uint4 raw4 = lds128_at(src + q * kPanelBytes + swizzled(t, at8));
              float x[8];
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.x), x[0], x[1]);
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.y), x[2], x[3]);
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.z), x[4], x[5]);
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.w), x[6], x[7]);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = t < n ? x[i] * w : 0.f;
              split3(x, hi, mid, lo);
              const uint32_t at = smem + kOffKp + (subs & 1) * kBlockBytes + q * kBlockPanel +
                                  swizzled(r, at8);
              sts128(at, hi[0], hi[1], hi[2], hi[3]);
              sts128(at + kBlockTile, mid[0], mid[1], mid[2], mid[3]);
              sts128(at + 2 * kBlockTile, lo[0], lo[1], lo[2], lo[3]);
            }
            cconv::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) cconv::mbar_arrive(&kpfull[subs & 1]);
          }
          if (!ok) break;
        }
        // rows of the output this thread finishes: row krow, columns [64 half, + 64)
        const float rowf = KV ? gt.kw[krow] : gt.er[krow];
        float dot = 0.f;
        if (KV && has) {
          if (!(ok = CATTN_WARP_WAIT(infull, pubs - 1))) break;
          if (!(ok = CATTN_WARP_WAIT(&full[kK], use))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // two batches of dk, two of dv
            const int col = half * 64 + (c & 1) * 32;
            const bool isk = c < 2;
            if (col < (isk ? p.K : vw)) {
              uint32_t x[32];
              const uint32_t at = tmem + lanes + (isk ? 256 : 384) + col;
              tmem_ld32(at, x);
              tmem_wait_ld();
              tmem_use32(x);
              if (isk) dot += dot_tile(ak, krow, col, x);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(rowf * __uint_as_float(x[i]));
              tmem_st16(at, x);
              tmem_st16(at + 16, x + 16);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) cconv::mbar_arrive(scaled);
        }
        if (KV) {
          if (!has && !(ok = CATTN_WARP_WAIT(scfull, use))) break;  // K Q^T reads the tile too
          __syncwarp();
          if (lane == 0) cconv::mbar_arrive(&empty[kK]);
        }
        if (flags & kNeedKv) {
          const float d = gt.total;
          if (!(ok = CATTN_WARP_WAIT(kvfull, kvs))) break;
          ++kvs;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld32(tmem + lanes + (KV ? half * 128 + 64 : 384 + half * 64) + c * 32, x);
            tmem_wait_ld();
            tmem_use32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              S[c * 32 + i] = fmaf(d, S[c * 32 + i], __uint_as_float(x[i]));
          }
          tc_fence_before();
          if (KV) {
            __syncwarp();
            if (lane == 0) cconv::mbar_arrive(kvfree);
          }
        }
        if (!(ok = CATTN_WARP_WAIT(ofull, use))) break;
        if (!KV && !(ok = CATTN_WARP_WAIT(&full[kQ], use))) break;
        tc_fence_after();
        const int hk = hv / p.ratio;
        const int64_t t = row0 + krow;
        float* prow = p.part ? p.part + (static_cast<int64_t>(ht) * p.rows + t) * p.K : nullptr;
        uint16_t* krow_out = (KV ? p.dk : p.dq) + (t * p.Hk + hk) * p.K;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = half * 64 + c * 32;
          if (col < p.K) {
            uint32_t x[32];
            tmem_ld32(tmem + lanes + (KV ? 256 : 128) + col, x);
            if (!KV && has) {
              uint32_t z[32];
              tmem_ld32(tmem + lanes + 256 + col, z);
              tmem_wait_ld();
              tmem_use32(x);
              tmem_use32(z);
              dot += dot_tile(aq, krow, col, z);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                x[i] = __float_as_uint(fmaf(rowf, __uint_as_float(z[i]), __uint_as_float(x[i])));
            } else {
              tmem_wait_ld();
              tmem_use32(x);
            }
            if (krow < n) {
              if (prow)
                store_f32(prow, col, p.K, x, p.scale);
              else
                store_bf16(krow_out, col, p.K, p.wide_k, x, p.scale);
            }
          }
        }
        if (KV) {
          uint16_t* vrow = p.dv + (t * p.Hv + hv) * p.V + vt * 128;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int col = half * 64 + c * 32;
            if (col < vw) {
              uint32_t x[32];
              tmem_ld32(tmem + lanes + 384 + col, x);
              tmem_wait_ld();
              tmem_use32(x);
              if (krow < n) store_bf16(vrow, col, vw, p.wide_v, x, p.scale);
            }
          }
        }
        if (krow < n)
          p.dots[(static_cast<int64_t>(1 + half) * p.plan.heads * p.plan.tiles + ht) * p.rows + t] =
              p.scale * rowf * dot;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!KV) cconv::mbar_arrive(&empty[kQ]);
          cconv::mbar_arrive(ofree);
        }
        ++use;
      }
      if (KV && (flags & kFinish) && krow < p.K) {
        float* dst = p.dinit + ((static_cast<int64_t>(gt.seq) * p.Hv + hv) * p.K + krow) * p.V +
                     vt * 128 + half * 64;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (half * 64 + 4 * i < vw)
            *reinterpret_cast<float4*>(dst + 4 * i) =
                make_float4(p.scale * S[4 * i], p.scale * S[4 * i + 1], p.scale * S[4 * i + 2],
                            p.scale * S[4 * i + 3]);
      }
      __syncwarp();
      if (lane == 0) cconv::mbar_arrive(&gempty[gs]);
    }
  }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

template <bool KV>
static int launch_sweep(const BwdArgs& a, int grid, cudaStream_t stream) {
  auto kern = cattn_linear_chunk_bwd_kernel<KV>;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kBwdBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(kern, dim3(grid), dim3(kBwdThreads), kBwdBytes, stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_chunk_bwd(const ChunkBwdCall& c, cudaStream_t stream) {
  BwdArgs a{};
  int rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mv, c.v, c.s.total, c.s.Hv, c.s.V);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mo, c.d_o, c.s.total, c.s.Hv, c.s.V);
  if (rc != CCONV_OK) return rc;
  a.plan = Plan{c.cu, c.cstart, c.s.nseq, (c.s.V + 127) / 128, c.s.Hv};
  a.g = c.g;
  a.slots = c.slots;
  a.initial = c.initial;
  a.dinit = c.dinit;
  a.dq = c.dq, a.dk = c.dk, a.dv = c.dv;
  a.scale = c.scale;
  a.rows = c.s.total, a.ratio = c.s.Hv / c.s.Hk;
  a.Hk = c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.wide_v = aligned(c.dv, 32) && c.s.V % 16 == 0;
  const bool even = c.s.K % 16 == 0;
  a.wide_k = even && aligned(c.dq, 32);
  a.carry = c.carry_s;
  a.decay = c.carry_s + static_cast<int64_t>(c.grid) * 2 * kStateFloats;
  a.part = c.part_q, a.dots = c.dots_q;
  rc = launch_sweep<false>(a, c.grid, stream);
  if (rc != CCONV_OK) return rc;
  a.wide_k = even && aligned(c.dk, 32);
  a.carry = c.carry_d;
  a.decay = c.carry_d + static_cast<int64_t>(c.grid) * 2 * kStateFloats;
  a.part = c.part_k, a.dots = c.dots_k;
  return launch_sweep<true>(a, c.grid, stream);
}

}  // namespace cattn
