// attn_chunk_fwd.cu -- linear attention with decay in chunks of 128 tokens on the tensor cores.
//
//   P = (Q K^T) . L,  L_ts = decay from s to t (s <= t)
//   o = scale * (P V + er . (Q S)),   S <- total S + (kw . K)^T V
//
// Two kernels over the same ranges of units (attn_chunk.cuh):
//   OUT = false  the state a range hands on: only the chunks since the last start of a sequence
//   OUT = true   the outputs; a range that starts inside a sequence sums the handed-on states
// The backward uses the first for the states and, with REV, for their gradients: the chunks
// from the last to the first, with (q, do) for (k, v) and er for kw.
//
// Roles of a CTA's 16 warps: one warp streams tiles by TMA through a ring of 32 KB slots, one
// thread issues every tcgen05.mma, one warp makes the gates; four warps turn scores into P and
// write o; eight warps keep the state.  Four matrix products a chunk (M = 128 each):
//   scores  Q K^T               -> TMEM [0, 128);  P overwrites it as bf16 and is the next A
//   P V                         -> TMEM [128, 256)
//   Q S                         -> TMEM [256, 384)
//   (kw . K)^T V                -> TMEM [384, 512)
// The state lives in registers in fp32 (64 columns of one row a thread).  Roundings to bf16: P
// and the copy of S that Q S reads, once each, and o at the store.  The products that build the
// state keep 24 bits of the decayed keys (three bf16 terms), so states stay accurate to fp32.
#include <cudaTypedefs.h>

#include <mutex>

#include "attn_chunk.cuh"
#include "attn_chunk_host.h"

namespace cattn {

static __device__ unsigned g_fault_fwd;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_fwd, sizeof(*out))) !=
          cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_fwd, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

constexpr int kStateWarps = 8;

template <bool OUT>
struct Layout {
  static constexpr int kTiles = OUT ? 3 : 2;   // tiles of a chunk: k, (q,) v
  static constexpr int kSlots = OUT ? 4 : 5;
  static constexpr int kOutWarps = OUT ? 4 : 0;
  static constexpr int kWarps = 4 + kOutWarps + kStateWarps;
  static constexpr int kThreads = kWarps * 32;
  // shared memory, from a 1024-byte boundary
  static constexpr int kRing = 0;
  static constexpr int kKp = kRing + kSlots * kTileBytes;      // two blocks of decayed keys
  static constexpr int kS = kKp + 2 * kSubBytes;               // the state in bf16
  static constexpr int kGates = kS + (OUT ? kTileBytes : 0);
  static constexpr int kBars = kGates + ((kGateStages * sizeof(Gate) + 15) / 16) * 16;
  static constexpr int kBytes = kBars + 40 * 8 + 1024;         // and the boundary's slack
};

struct ChunkArgs {
  CUtensorMap mq, mk, mv;
  Plan plan;
  Gates g;
  Slots slots;
  const float* initial;
  float* fin;
  const int32_t* status;
  uint16_t* o;
  float* carry;   // [grid] states handed on
  float* decay;   // [grid] their decays; negative: the sequence began in that range
  float* copy;    // [grid] initial states of split sequences (final_state may overwrite them)
  float scale;
  int rows, ratio, Hv, K, V;
  int wide;       // o's rows allow 32-byte stores
};

#define CATTN_WAIT(bar, parity)                                        \
  (wait_phase((bar), static_cast<uint32_t>(parity) & 1u, gave_up, &g_fault_fwd))
#define CATTN_WARP_WAIT(bar, parity) (__all_sync(0xffffffffu, CATTN_WAIT(bar, parity)))

template <bool OUT, bool REV>
__global__ void __launch_bounds__(Layout<OUT>::kThreads, 1)
    cattn_linear_chunk_kernel(const __grid_constant__ ChunkArgs p) {
  using L = Layout<OUT>;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Gate* gates = reinterpret_cast<Gate*>(base + L::kGates);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::kBars);
  uint64_t *full = bars, *empty = bars + L::kSlots;
  uint64_t *gfull = empty + L::kSlots, *gempty = gfull + kGateStages;
  uint64_t *kpfull = gempty + kGateStages, *kpempty = kpfull + 2;
  uint64_t *kvfull = kpempty + 2, *vfixed = kvfull + 1, *scfull = vfixed + 2, *pfull = scfull + 1;
  uint64_t *ofull = pfull + 1, *ofree = ofull + 1, *sfull = ofree + 1, *sempty = sfull + 1;
  uint64_t* alldone = sempty + 1;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(alldone + 1);
  volatile int* gave_up = reinterpret_cast<int*>(tmem_at + 1);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      cconv::mbar_init(&full[i], 1);
      cconv::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kGateStages; ++i) {
      cconv::mbar_init(&gfull[i], 1);
      cconv::mbar_init(&gempty[i], L::kOutWarps + kStateWarps + 1);
    }
    for (int i = 0; i < 2; ++i) {
      cconv::mbar_init(&kpfull[i], kStateWarps);
      cconv::mbar_init(&kpempty[i], 1);
      cconv::mbar_init(&vfixed[i], kStateWarps);
    }
    cconv::mbar_init(kvfull, 1);
    cconv::mbar_init(scfull, 1);
    cconv::mbar_init(pfull, 4);
    cconv::mbar_init(ofull, 1);
    cconv::mbar_init(ofree, 4);
    cconv::mbar_init(sfull, kStateWarps);
    cconv::mbar_init(sempty, 1);
    cconv::mbar_init(alldone, 1);
    *gave_up = 0;
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_at, 512);
  if (warp == 0 && lane == 0 && p.rows > 0) {
    cconv::prefetch_tensormap(&p.mk);
    cconv::prefetch_tensormap(&p.mv);
    if (OUT) cconv::prefetch_tensormap(&p.mq);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const uint32_t smem = smem_addr(base);
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();

  // The CTA's units.
  int nch;
  const int64_t units = unit_count(p.plan, nch);
  const int64_t parts = min(static_cast<int64_t>(gridDim.x), units);
  Range range{0, 0};
  if (blockIdx.x < parts) range = range_of(units, parts, blockIdx.x);
  const Tail tail = tail_of<REV>(p.plan, nch, units, range);
  if (!OUT) range = Range{tail.u0, tail.u1};  // nothing else is handed on
  const int64_t count = range.u1 - range.u0, start = REV ? range.u1 - 1 : range.u0;
  const int pk = p.K > kPanelCols ? 2 : 1;

  if (count > 0) {
  if (warp == 0) {
    // ---- tiles ----
    if (lane == 0) {
      Walker w;
      w.seek(&p.plan, nch, start);
      int tile = 0;
      bool ok = true;
      for (int64_t i = 0; i < count && ok; ++i) {
        if (w.rows() > 0) {
          const int hv = w.ht / p.plan.tiles, vt = w.ht % p.plan.tiles;
          const int hk = hv / p.ratio, row = w.row0();
          const int pv = p.V - vt * 128 > kPanelCols ? 2 : 1;
          for (int j = 0; j < L::kTiles && ok; ++j, ++tile) {
            const int slot = tile % L::kSlots, use = tile / L::kSlots;
            if (use > 0 && !(ok = CATTN_WAIT(&empty[slot], use - 1))) break;
            const bool isv = j == L::kTiles - 1;
            const CUtensorMap* map = isv ? &p.mv : j == 0 ? &p.mk : &p.mq;
            const int panels = isv ? pv : pk;
            uint8_t* dst = base + L::kRing + slot * kTileBytes;
            cconv::mbar_arrive_expect_tx(&full[slot], panels * kPanelBytes);
            for (int c = 0; c < panels; ++c)
              cconv::tma_load_3d(dst + c * kPanelBytes, map, &full[slot],
                                 (isv ? vt * 128 : 0) + c * kPanelCols, isv ? hv : hk, row);
          }
        }
        if (i + 1 < count) w.step<REV>();
      }
      cconv::drain_issued<L::kSlots>(full, tile);
    }
  } else if (warp == 1) {
    // ---- matrix products ----
    if (lane == 0) {
      int tile = 0, unit = 0, scs = 0, subs = 0, fixes = 0, pubs = 0;
      bool ok = true;
      const uint32_t ring = smem + L::kRing;
      const int ksteps = (p.K + 15) / 16;
      const uint32_t d_scores = mma_desc(128, false, false);
      for (; unit < count && ok; ++unit) {
        const int gs = unit % kGateStages;
        if (!(ok = CATTN_WAIT(&gfull[gs], unit / kGateStages))) break;
        const Gate& gt = gates[gs];
        const int n = gt.n, flags = gt.flags, ht = gt.ht;
        if (n > 0) {
          const int vw = min(128, p.V - ht % p.plan.tiles * 128);
          const int nv = (vw + 15) / 16 * 16;
          const int tk = tile, tq = tile + 1, tv = tile + L::kTiles - 1;
          tile += L::kTiles;
          const uint32_t ak = ring + tk % L::kSlots * kTileBytes;
          const uint32_t aq = ring + tq % L::kSlots * kTileBytes;
          const uint32_t av = ring + tv % L::kSlots * kTileBytes;
          if (!(ok = CATTN_WAIT(&full[tk % L::kSlots], tk / L::kSlots))) break;
          if (OUT) {
            if (!(ok = CATTN_WAIT(&full[tq % L::kSlots], tq / L::kSlots))) break;
            // the scores overwrite the last chunk's P, which P V must have read
            if (scs > 0 && !(ok = CATTN_WAIT(ofull, scs - 1))) break;
            tc_fence_after();
            for (int j = 0; j < ksteps; ++j) {
              const uint32_t off = (j / 4) * kPanelBytes + (j % 4) * 32;
              mma_ss(tmem, tile_desc(aq + off, 0), tile_desc(ak + off, 0), d_scores, j > 0);
            }
            mma_commit(scfull);
            if (scs > 0 && !(ok = CATTN_WAIT(ofree, scs - 1))) break;
            tc_fence_after();
            if (flags & kHasState) {
              if (!(ok = CATTN_WAIT(sfull, pubs))) break;
              ++pubs;
              tc_fence_after();
              const uint32_t d = mma_desc(nv, false, true);
              for (int j = 0; j < ksteps; ++j)
                mma_ss(tmem + 256, tile_desc(aq + (j / 4) * kPanelBytes + (j % 4) * 32, 0),
                       tile_desc(smem + L::kS + j * 2048, kPanelBytes), d, j > 0);
              mma_commit(sempty);
            }
            mma_commit(&empty[tq % L::kSlots]);
          }
          if (!(ok = CATTN_WAIT(&full[tv % L::kSlots], tv / L::kSlots))) break;
          if (n < kChunk) {
            if (!(ok = CATTN_WAIT(&vfixed[fixes & 1], fixes >> 1))) break;
            ++fixes;
          }
          if (flags & kNeedKv) {
            const uint32_t d = mma_desc(nv, true, true);
            const int blocks = (n + kSub - 1) / kSub;
            for (int b = 0; b < blocks; ++b, ++subs) {
              if (!(ok = CATTN_WAIT(&kpfull[subs & 1], subs >> 1))) break;
              tc_fence_after();
              for (int s = 0; s < kSplit; ++s)
                for (int j = 0; j < 2; ++j)
                  mma_ss(tmem + 384,
                         tile_desc(smem + L::kKp + (subs & 1) * kSubBytes + s * kSubTile + j * 2048,
                                   kSubPanel),
                         tile_desc(av + (b * 2 + j) * 2048, kPanelBytes), d, b + s + j > 0);
              mma_commit(&kpempty[subs & 1]);
            }
            if (!ok) break;
            mma_commit(kvfull);
          }
          mma_commit(&empty[tk % L::kSlots]);
          if (OUT) {
            if (!(ok = CATTN_WAIT(pfull, scs))) break;
            ++scs;
            tc_fence_after();
            const uint32_t d = mma_desc(nv, false, true);
            const int steps = (n + 15) / 16;
            for (int j = 0; j < steps; ++j)
              mma_ts(tmem + 128, tmem + j * 8, tile_desc(av + j * 2048, kPanelBytes), d, j > 0);
            mma_commit(ofull);
          }
          mma_commit(&empty[tv % L::kSlots]);
        }
        cconv::mbar_arrive(&gempty[gs]);
      }
      // nothing of this CTA may be in flight when its shared memory and TMEM go
      mma_commit(alldone);
      (void)cconv::mbar_wait_bounded(alldone, 0, cconv::kDrainLimitNs);
    }
  } else if (warp == 2) {
    // ---- gates ----
    Walker w;
    w.seek(&p.plan, nch, start);
    for (int64_t i = 0; i < count; ++i) {
      const int unit = static_cast<int>(i);
      const int gs = unit % kGateStages, n = w.rows(), row0 = w.row0();
      const int hv = w.ht / p.plan.tiles;
      float g[4];
#pragma unroll
      for (int b = 0; b < 4; ++b)
        g[b] = 32 * b + lane < n ? kLog2e * p.g.at(row0 + 32 * b + lane, hv) : 0.f;
      if (unit >= kGateStages && !CATTN_WARP_WAIT(&gempty[gs], unit / kGateStages - 1)) break;
      Gate& gt = gates[gs];
      make_gate(gt, g, lane);
      if (lane == 0) {
        gt.row0 = row0;
        gt.n = n;
        gt.ht = w.ht;
        gt.seq = w.seq;
        int f = 0;
        const bool first = REV ? w.last() : w.first();
        if (i == 0 || first) f |= kSegment;
        if ((f & kSegment) && !first) f |= kMiddle;
        if (!first || p.initial) f |= kHasState;
        if (w.last() && p.fin && OUT) f |= kFinish;
        if (OUT ? (!w.last() && i + 1 < count) || (f & kFinish) : true) f |= kNeedKv;
        if (range.u0 + i >= tail.u0 && tail.closed) f |= kSplitSeq;
        gt.flags = f;
      }
      __syncwarp();
      if (lane == 0) cconv::mbar_arrive(&gfull[gs]);
      if (i + 1 < count) w.step<REV>();
    }
  } else if (OUT && warp >= 4 && warp < 8) {
    // ---- scores to P, and the outputs ----
    const int wq = warp - 4, row = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    int scs = 0;
    for (int unit = 0; unit < count; ++unit) {
      const int gs = unit % kGateStages;
      if (!CATTN_WARP_WAIT(&gfull[gs], unit / kGateStages)) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, row0 = gt.row0, ht = gt.ht;
      const bool inter = gt.flags & kHasState;
      const float er = gt.er[row];
      if (n > 0) {
        if (!CATTN_WARP_WAIT(scfull, scs)) break;
        tc_fence_after();
        const float lp = gt.lp[row];
        for (int b = 0; b < 4; ++b) {
          uint32_t x[32], y[16];
          if (b <= wq) {
            tmem_ld32(tmem + lanes + b * 32, x);
            tmem_wait_ld();
            tmem_use32(x);
          }
          if (b < wq) {
            float e = lp;
            for (int i = b + 1; i < wq; ++i) e += gt.block[i];
            const float ut = exp2_fast(e);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 ws = *reinterpret_cast<const float4*>(&gt.ws[b * 32 + i * 4]);
              y[2 * i] = pack_bf16(__uint_as_float(x[4 * i]) * (ut * ws.x),
                                   __uint_as_float(x[4 * i + 1]) * (ut * ws.y));
              y[2 * i + 1] = pack_bf16(__uint_as_float(x[4 * i + 2]) * (ut * ws.z),
                                       __uint_as_float(x[4 * i + 3]) * (ut * ws.w));
            }
          } else if (b == wq) {
            // the diagonal block: the decay from s to t as a running product down from t
            float w = 1.f, hi = 0.f;
#pragma unroll
            for (int s = 31; s >= 0; --s) {
              if (s < lane) w *= gt.a[b * 32 + s + 1];
              const float v = s <= lane ? __uint_as_float(x[s]) * w : 0.f;
              if (s & 1)
                hi = v;
              else
                y[s / 2] = pack_bf16(v, hi);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = 0;
          }
          tmem_st16(tmem + lanes + b * 16, y);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cconv::mbar_arrive(pfull);
        if (!CATTN_WARP_WAIT(ofull, scs)) break;
        ++scs;
        tc_fence_after();
        const int vt = ht % p.plan.tiles, vw = min(128, p.V - vt * 128);
        uint16_t* dst = p.o + (static_cast<int64_t>(row0 + row) * p.Hv + ht / p.plan.tiles) * p.V +
                        vt * 128;
        const float es = p.scale * er;
        for (int c = 0; c < vw; c += 32) {
          uint32_t x[32], z[32], y[16];
          tmem_ld32(tmem + lanes + 128 + c, x);
          if (inter) tmem_ld32(tmem + lanes + 256 + c, z);
          tmem_wait_ld();
          tmem_use32(x);
          if (inter) {
            tmem_use32(z);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = __float_as_uint(
                  fmaf(es, __uint_as_float(z[i]), p.scale * __uint_as_float(x[i])));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(p.scale * __uint_as_float(x[i]));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            y[i] = pack_bf16(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
          if (row < n) {
            if (p.wide && c + 32 <= vw) {
              stg256(dst + c, y);
              stg256(dst + c + 16, y + 8);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (c + 8 * i < vw)
                  *reinterpret_cast<uint4*>(dst + c + 8 * i) =
                      make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cconv::mbar_arrive(ofree);
      }
      __syncwarp();
      if (lane == 0) cconv::mbar_arrive(&gempty[gs]);
    }
  } else if (warp >= 4 + L::kOutWarps) {
    // ---- the state ----
    const int st = threadIdx.x - (4 + L::kOutWarps) * 32;  // 0 .. 255
    const int half = st / 128, krow = st % 128;            // columns [64 half, 64 half + 64) of row
    const uint32_t lanes = static_cast<uint32_t>(krow & ~31) << 16;
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    float passed = 1.f;  // decay of the chunks so far (what is handed on)
    int tile = 0, unit = 0, kvs = 0, subs = 0, pubs = 0, fixes = 0;
    bool ok = true;
    for (; unit < count && ok; ++unit) {
      const int gs = unit % kGateStages;
      if (!(ok = CATTN_WARP_WAIT(&gfull[gs], unit / kGateStages))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, flags = gt.flags, ht = gt.ht;
      const int hv = ht / p.plan.tiles, vt = ht % p.plan.tiles;
      const int vw = min(128, p.V - vt * 128);
      const int64_t slot = p.slots.of(gt.seq);
      if (flags & kSegment) {
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0.f;
        if (flags & kMiddle) {
          if (OUT) {
            // what the ranges before this one hand on, back to the one where the sequence began
            float coef = 1.f;
            for (int64_t j = blockIdx.x - 1; j >= 0; --j) {
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
          }
        } else if (p.initial && slot >= 0 && krow < p.K) {
          const bool saved = OUT && (flags & kSplitSeq) && p.fin;
          const float* src = p.initial + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128 + half * 64;
          const float4* from = reinterpret_cast<const float4*>(p.copy + static_cast<int64_t>(blockIdx.x) * kStateFloats);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (saved)
              x = from[(half * 16 + i) * 128 + krow];
            else if (half * 64 + 4 * i < vw)
              x = *reinterpret_cast<const float4*>(src + 4 * i);
            S[4 * i] = x.x, S[4 * i + 1] = x.y, S[4 * i + 2] = x.z, S[4 * i + 3] = x.w;
          }
        }
        if (!OUT && tail.closed && p.initial && p.fin) {
          // the outputs' kernel reads this copy: by then final_state may have replaced it
          float4* to = reinterpret_cast<float4*>(p.copy + static_cast<int64_t>(blockIdx.x) * kStateFloats);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            to[(half * 16 + i) * 128 + krow] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
      }
      if (OUT && n > 0 && (flags & kHasState)) {
        if (pubs > 0 && !(ok = CATTN_WARP_WAIT(sempty, pubs - 1))) break;
        ++pubs;
        const uint32_t dst = smem + L::kS + half * kPanelBytes;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          sts128(dst + swizzled(krow, i), pack_bf16(S[8 * i], S[8 * i + 1]),
                 pack_bf16(S[8 * i + 2], S[8 * i + 3]), pack_bf16(S[8 * i + 4], S[8 * i + 5]),
                 pack_bf16(S[8 * i + 6], S[8 * i + 7]));
        cconv::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) cconv::mbar_arrive(sfull);
      }
      if (n > 0) {
        const int tk = tile, tv = tile + L::kTiles - 1;
        tile += L::kTiles;
        if (n < kChunk) {
          if (!(ok = CATTN_WARP_WAIT(&full[tv % L::kSlots], tv / L::kSlots))) break;
          zero_rows(smem + L::kRing + tv % L::kSlots * kTileBytes, vw > kPanelCols ? 2 : 1, n, st,
                    kStateWarps * 32);
          cconv::fence_proxy_async_smem();
          __syncwarp();
          // (chunks that need no state let these warps run one chunk ahead of the products:
          // two barriers in turn)
          if (lane == 0) cconv::mbar_arrive(&vfixed[fixes & 1]);
          ++fixes;
        }
        if (flags & kNeedKv) {
          if (!(ok = CATTN_WARP_WAIT(&full[tk % L::kSlots], tk / L::kSlots))) break;
          const uint32_t src = smem + L::kRing + tk % L::kSlots * kTileBytes;
          const int r = st / 8, piece = st % 8;  // one token's 16-byte pieces `piece` of each panel
          const int blocks = (n + kSub - 1) / kSub;
          for (int b = 0; b < blocks; ++b, ++subs) {
            if (subs >= 2 && !(ok = CATTN_WARP_WAIT(&kpempty[subs & 1], (subs >> 1) - 1))) break;
            const int t = b * kSub + r;
            const float w = REV ? gt.er[t] : gt.kw[t];
            const uint32_t dst = smem + L::kKp + (subs & 1) * kSubBytes;
            for (int q = 0; q < pk; ++q) {
              uint32_t hi[4], mid[4], lo[4];
              const uint4 raw4 = lds128_at(src + q * kPanelBytes + swizzled(t, piece));
              float x[8];
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.x), x[0], x[1]);
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.y), x[2], x[3]);
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.z), x[4], x[5]);
              cconv::f2_unpack(cconv::bf16x2_to_f2(raw4.w), x[6], x[7]);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = t < n ? x[i] * w : 0.f;
              split3(x, hi, mid, lo);
              const uint32_t at = dst + q * kSubPanel + swizzled(r, piece);
              sts128(at, hi[0], hi[1], hi[2], hi[3]);
              sts128(at + kSubTile, mid[0], mid[1], mid[2], mid[3]);
              sts128(at + 2 * kSubTile, lo[0], lo[1], lo[2], lo[3]);
            }
            cconv::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) cconv::mbar_arrive(&kpfull[subs & 1]);
          }
          if (!ok) break;
          const float d = gt.total;
          if (!(ok = CATTN_WARP_WAIT(kvfull, kvs))) break;
          ++kvs;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[32];
            tmem_ld32(tmem + lanes + 384 + half * 64 + c * 32, x);
            tmem_wait_ld();
            tmem_use32(x);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              S[c * 32 + i] = fmaf(d, S[c * 32 + i], __uint_as_float(x[i]));
          }
          tc_fence_before();
          passed *= d;
        }
      }
      if ((flags & kFinish) && slot >= 0 && krow < p.K && !(p.status && p.status[0] != CCONV_OK)) {
        float* dst = p.fin + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128 + half * 64;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (half * 64 + 4 * i < vw)
            *reinterpret_cast<float4*>(dst + 4 * i) =
                make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
      }
      __syncwarp();
      if (lane == 0) cconv::mbar_arrive(&gempty[gs]);
    }
    if (!OUT && ok) {
      float4* to = reinterpret_cast<float4*>(p.carry + static_cast<int64_t>(blockIdx.x) * kStateFloats);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        to[(half * 16 + i) * 128 + krow] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
      if (st == 0) p.decay[blockIdx.x] = tail.closed ? -1.f : passed;
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

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Map of a [total, H, C] tensor read in boxes of 64 channels of one head and 128 tokens.
int encode_tile_map(CUtensorMap* map, const Rows& x, int64_t total, int64_t H, int64_t C) {
  auto enc = encode_fn();
  if (!enc) return CCONV_ERR_CUDA;
  // strides over dimensions of extent 1 are the caller's to leave unset
  const int64_t sh = H > 1 ? x.sh : C, st = total > 1 ? x.st : C * H;
  cuuint64_t dims[3] = {(cuuint64_t)C, (cuuint64_t)H, (cuuint64_t)total};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2u, (cuuint64_t)st * 2u};
  cuuint32_t box[3] = {kPanelCols, 1u, kChunk};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(x.p), dims, strides, box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CCONV_OK : CCONV_ERR_CUDA;
}

template <bool OUT, bool REV>
static int launch(const ChunkArgs& a, int grid, cudaStream_t stream) {
  using L = Layout<OUT>;
  auto kern = cattn_linear_chunk_kernel<OUT, REV>;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), L::kBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(kern, dim3(grid), dim3(L::kThreads), L::kBytes, stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

int launch_chunk_fwd(const ChunkCall& c, cudaStream_t stream) {
  ChunkArgs a{};
  int rc = CCONV_OK;
  if (c.s.total > 0) {
    rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K);
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K);
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mv, c.v, c.s.total, c.s.Hv, c.s.V);
    if (rc != CCONV_OK) return rc;
  }
  const int tiles = (c.s.V + 127) / 128;
  a.plan = Plan{c.cu, c.cstart, c.s.nseq, tiles, c.s.Hv};
  a.g = c.g;
  a.slots = c.slots;
  a.initial = c.initial;
  a.fin = c.fin;
  a.status = c.status;
  a.o = c.o;
  a.carry = c.carry;
  a.copy = c.carry + static_cast<int64_t>(c.grid) * kStateFloats;
  a.decay = a.copy + static_cast<int64_t>(c.grid) * kStateFloats;
  a.scale = c.scale;
  a.rows = c.s.total;
  a.ratio = c.s.Hv / c.s.Hk;
  a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.wide = aligned(c.o, 32) && c.s.V % 16 == 0;
  if (c.part == kStates) return launch<false, false>(a, c.grid, stream);
  if (c.part == kStateGrads) return launch<false, true>(a, c.grid, stream);
  rc = launch<false, false>(a, c.grid, stream);
  return rc == CCONV_OK ? launch<true, false>(a, c.grid, stream) : rc;
}

size_t chunk_fwd_bytes(int grid) {
  return static_cast<size_t>(grid) * (2 * kStateFloats + 4) * sizeof(float);
}

}  // namespace cattn
