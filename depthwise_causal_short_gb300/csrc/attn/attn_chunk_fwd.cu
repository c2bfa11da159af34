// attn_chunk_fwd.cu -- linear attention with decay in chunks of 128 tokens on the tensor cores.
//
//   P = (Q K^T) . L,  L_ts = decay from s to t (s <= t)
//   o = scale * (P V + er . (Q S)),   S <- total S + (kw . K)^T V
//
// Two kernels over the same ranges of units (attn_chunk.cuh): cattn_linear_tail_kernel computes
// the state that each range hands on, cattn_linear_chunk_kernel the outputs; a range that starts
// inside a sequence sums the handed-on states.  cattn_linear_tails_kernel is the backward's first:
// the states and, with REV, their gradients: (q, do) for (k, v), decays to the range's start.
//
// Roles of a CTA's 16 warps: one warp streams tiles by TMA through a ring of 32 KB slots, one
// thread issues the products of the outputs and one those of the state, one warp makes the
// gates; four warps turn scores into P and write o; four make the
// decayed keys; four keep the state.  Outputs and state advance independently, up to the ring's
// depth.  Four matrix products a chunk (M = 128 each):
//   scores  Q K^T               -> TMEM [0, 128);  P overwrites it as bf16 and is the next A
//   P V                         -> TMEM [128, 256)
//   Q S                         -> TMEM [256, 384)
//   (kw . K)^T V                -> TMEM [384, 512)
// The state lives in registers in fp32 (one row a thread).  Roundings to bf16: P
// and the copy of S that Q S reads, once each, and o at the store.  The products that build the
// state keep 24 bits of the decayed keys (three bf16 terms), so states stay accurate to fp32.
//
// Bound by the chain of the roles within a chunk: its 48 products of 128 x 128 x 16 are 3000 cycles of
// the tensor cores, which with the warps' accesses keep shared memory busy for 4700; it takes 8000
// (tensor cores active 25 % of the time, load / store unit 29 %, DRAM 40 %).  16384 rows in 2
// sequences, 16 value heads on 8 key heads of 128: 110 us (37 of them the states handed on), 1.8 TB/s
// of needed bytes; one chunk 7.5 us.  Two slots for v and one for k took as long as one and two; tiles
// fetched to L2 ahead 1 % longer.
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

enum FwdSlot : int { kKeys0 = 0, kKeys1 = 1, kQuery = 2, kValue = 3, kSlots = 4 };  // k in turn
constexpr int kKeyWarps = 4;
constexpr int kReaders = 4 + kKeyWarps + 4 + 2;  // warps that read a gate
constexpr int kFwdThreads = 512;
// shared memory, from a 1024-byte boundary
constexpr int kOffKp = kSlots * kTileBytes;        // two blocks of decayed keys
constexpr int kOffS = kOffKp + 2 * kSubBytes;      // the state in bf16; a chunk's outputs
constexpr int kOffGates = kOffS + kTileBytes;
constexpr int kOffBars = kOffGates + kGateStages * sizeof(Gate);
constexpr int kFwdBytes = kOffBars + 40 * 8 + 1024;  // and the boundary's slack
static_assert(kFwdBytes <= 232448, "shared memory of one CTA");

struct ChunkArgs {
  CUtensorMap mq, mk, mv, mo;
  Plan plan;
  Gates g;
  Slots slots;
  const float* initial;
  float* fin;
  uint16_t* o;
  float* carry;   // [grid] states handed on
  float* decay;   // [grid] their decays, kChainStart or kNoTail
  float* copy;    // [grid] initial states of split sequences (final_state may overwrite them)
  float scale;
  int rows, ratio, Hv, K, V;
  int joined;     // the states handed on are whole (the scan kernel ran)
  int report;     // the tail kernel writes a small plan's verdicts (the backward's first)
};

#define CATTN_WAIT(bar, parity) (wait_phase((bar), static_cast<uint32_t>(parity) & 1u))
#define CATTN_WARP_WAIT(bar, parity) (__all_sync(0xffffffffu, CATTN_WAIT(bar, parity)))

template <bool FINE>
__global__ void __launch_bounds__(kFwdThreads, 1)
    cattn_linear_chunk_kernel(const __grid_constant__ ChunkArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Gate* gates = reinterpret_cast<Gate*>(base + kOffGates);
  const uint32_t smem = smem_addr(base);
  // barriers, 8 bytes each
  const uint32_t full = smem + kOffBars, empty = full + 8 * kSlots;
  const uint32_t gfull = empty + 8 * kSlots, gempty = gfull + 8 * kGateStages;
  const uint32_t kpfull = gempty + 8 * kGateStages, kpempty = kpfull + 16, vfixed = kpempty + 16;
  const uint32_t kvfull = vfixed + 8, kvfree = kvfull + 8, scfull = kvfree + 8, pfull = scfull + 8;
  const uint32_t ofull = pfull + 8, ofree = ofull + 8, sfull = ofree + 8, sempty = sfull + 8;
  const uint32_t osync = sempty + 8, alldone = osync + 8;  // one for each issuing thread
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(base + kOffBars + 39 * 8);
  const uint32_t stored = smem + kOffBars + 38 * 8;  // chunks whose outputs have left the buffer

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      bar_init(full + 8 * (i), 1);
      // readers: the outputs' products; for k the warps that make decayed keys, for v the state's
      // products
      bar_init(empty + 8 * (i), i == kQuery ? 1 : i == kValue ? 2 : 1 + kKeyWarps);
    }
    for (int i = 0; i < kGateStages; ++i) {
      bar_init(gfull + 8 * (i), 1);
      bar_init(gempty + 8 * (i), kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(kpfull + 8 * (i), kKeyWarps);
      bar_init(kpempty + 8 * (i), 1);
      bar_init(alldone + 8 * (i), 1);
    }
    bar_init(vfixed, 4);
    bar_init(kvfull, 1);
    bar_init(kvfree, 4);
    bar_init(scfull, 1);
    bar_init(pfull, 4);
    bar_init(ofull, 1);
    bar_init(ofree, 4);
    bar_init(sfull, 4);
    bar_init(sempty, 1);
    set_count(stored, 0);
    bar_init(osync, 4);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_at, 512);
  if (warp == 0 && lane == 0 && p.rows > 0) {
    cconv::prefetch_tensormap(&p.mk);
    cconv::prefetch_tensormap(&p.mv);
    cconv::prefetch_tensormap(&p.mq);
    cconv::prefetch_tensormap(&p.mo);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ SmallPlan small;
  Plan plan = p.plan;
  if (plan.small) small_plan(plan, small, blockIdx.x == 0, &g_fault_fwd);

  // The CTA's units.
  int nch;
  const int64_t units = unit_count(plan, nch);
  const int64_t parts = min(static_cast<int64_t>(gridDim.x), units);
  Range range{0, 0};
  if (blockIdx.x < parts) range = range_of(units, parts, blockIdx.x);
  const Tail tail = tail_of<false>(plan, nch, units, range);
  const int64_t count = range.u1 - range.u0;
  const int pk = p.K > kPanelCols ? 2 : 1;

  bool ok = true;  // no wait of this thread's has given up
  if (count > 0) {
  if (warp < 4) {
  // Registers: 128 a thread at the launch, 56 + 128 + 104 + 208 after.
  set_registers<56, false>();
  if (warp == 0) {
    // ---- tiles ----
    if (elect_one()) {
      Walker w;
      w.seek(&plan, nch, range.u0);
      int chunk = 0, part = 0;
      for (int64_t i = 0; i < count && ok; ++i) {
        if (w.rows() > 0) {
          const int hv = w.ht / plan.tiles, vt = w.ht % plan.tiles;
          const int hk = hv / p.ratio, row = w.row0();
          const int pv = p.V - vt * 128 > kPanelCols ? 2 : 1;
#pragma unroll 1
          for (int j = 0; j < 3 && ok; ++j) {
            const int slot = j == 0 ? chunk & 1 : j + 1, use = j == 0 ? chunk >> 1 : chunk;
            if (use > 0 && !(ok = CATTN_WAIT(empty + 8 * (slot), use - 1))) break;
            part = j + 1;
            const bool isv = j == 2;
            const CUtensorMap* map = isv ? &p.mv : j == 0 ? &p.mk : &p.mq;
            const int panels = isv ? pv : pk;
            const uint32_t dst = smem + slot * kTileBytes;
            bar_expect(full + 8 * (slot), panels * kPanelBytes);
#pragma unroll 1
            for (int c = 0; c < panels; ++c)
              load_box(dst + c * kPanelBytes, map, full + 8 * slot,
                                 (isv ? vt * 128 : 0) + c * kPanelCols, isv ? hv : hk, row);
          }
          if (!ok) break;
          ++chunk;
          part = 0;
        }
        if (i + 1 < count) w.next();
      }
      // loads into the slots, those of a chunk that gave up half-way among them
      drain(full + 8 * kKeys0, (chunk + 1 + (part > 0)) / 2);
      drain(full + 8 * kKeys1, (chunk + (part > 0)) / 2);
      drain(full + 8 * kQuery, chunk + (part > 1));
      drain(full + 8 * kValue, chunk + (part > 2));
    }
  } else if (warp == 1) {
    // ---- scores, Q S and P V ----
    if (elect_one()) {
      int scs = 0, pubs = 0;
      const int ksteps = (p.K + 15) / 16;
      const uint64_t dq = tile_desc(smem + kQuery * kTileBytes, 0);
      const uint64_t dv = tile_desc(smem + kValue * kTileBytes, kPanelBytes);
      const uint64_t ds = tile_desc(smem + kOffS, kPanelBytes);
      const uint32_t d_scores = mma_desc(128, false, false);
      for (int unit = 0; unit < count && ok; ++unit) {
        const int gs = unit % kGateStages;
        if (!(ok = CATTN_WAIT(gfull + 8 * (gs), unit / kGateStages))) break;
        const Gate& gt = gates[gs];
        const int n = gt.n, flags = gt.flags;
        if (n > 0) {
          const int nv = (min(128, p.V - gt.ht % plan.tiles * 128) + 15) / 16 * 16;
          const uint32_t d_out = mma_desc(nv, false, true);
          const int key = scs & 1;
          if (!(ok = CATTN_WAIT(full + 8 * key, scs >> 1))) break;
          if (!(ok = CATTN_WAIT(full + 8 * kQuery, scs))) break;
          // the scores overwrite the last chunk's P, which P V must have read
          if (scs > 0 && !(ok = CATTN_WAIT(ofull, scs - 1))) break;
          tc_fence_after();
          const uint64_t dk = tile_desc(smem + key * kTileBytes, 0);
#pragma unroll 1
          for (int j = 0; j < ksteps; ++j)
            mma_ss(tmem, dq + col_step(j), dk + col_step(j), d_scores, j > 0);
          mma_commit(scfull);
          mma_commit(empty + 8 * key);
          if (scs > 0 && !(ok = CATTN_WAIT(ofree, scs - 1))) break;
          tc_fence_after();
          if (flags & kHasState) {
            if (!(ok = CATTN_WAIT(sfull, pubs))) break;
            ++pubs;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < ksteps; ++j)
              mma_ss(tmem + 256, dq + col_step(j), ds + j * kRowStep, d_out, j > 0);
            mma_commit(sempty);
          }
          mma_commit(empty + 8 * kQuery);
          if (!(ok = CATTN_WAIT(full + 8 * kValue, scs))) break;
          if (!(ok = CATTN_WAIT(pfull, scs))) break;
          ++scs;
          tc_fence_after();
          mma_p<FINE>(tmem + 128, tmem, dv, d_out, (n + 15) / 16, false);
          mma_commit(ofull);
          mma_commit(empty + 8 * kValue);
        }
        bar_arrive(gempty + 8 * (gs));
      }
      // nothing of this CTA may be in flight when its shared memory and TMEM go
      mma_commit(alldone + 8 * (0));
      drain(alldone + 8 * (0), 1);
    }
  } else if (warp == 3) {
    // ---- (kw . K)^T V ----
    if (elect_one()) {
      int chunk = 0, subs = 0, fixes = 0, kvs = 0;
      const uint32_t av = smem + kValue * kTileBytes;
      for (int unit = 0; unit < count && ok; ++unit) {
        const int gs = unit % kGateStages;
        if (!(ok = CATTN_WAIT(gfull + 8 * (gs), unit / kGateStages))) break;
        const Gate& gt = gates[gs];
        const int n = gt.n, flags = gt.flags;
        if (n > 0) {
          const int nv = (min(128, p.V - gt.ht % plan.tiles * 128) + 15) / 16 * 16;
          if (!(ok = CATTN_WAIT(full + 8 * kValue, chunk))) break;
          if (n < kChunk && !(ok = CATTN_WAIT(vfixed, fixes++))) break;
          ++chunk;
          if (flags & kNeedKv) {
            if (kvs > 0 && !(ok = CATTN_WAIT(kvfree, kvs - 1))) break;
            const uint32_t d = mma_desc(nv, true, true);
            const int blocks = (n + kSub - 1) / kSub;
#pragma unroll 1
            for (int b = 0; b < blocks; ++b, ++subs) {
              if (!(ok = CATTN_WAIT(kpfull + 8 * (subs & 1), subs >> 1))) break;
              tc_fence_after();
              const uint64_t da = tile_desc(smem + kOffKp + (subs & 1) * kSubBytes, kSubPanel);
              const uint64_t db = tile_desc(av + b * kSub * 128, kPanelBytes);
#pragma unroll 1
              for (int s = 0; s < 2 * kSplit; ++s)  // term s / 2, tokens [16 (s & 1), + 16)
                mma_ss(tmem + 384, da + (s >> 1) * (kSubTile / 16) + (s & 1) * kRowStep,
                       db + (s & 1) * kRowStep, d, b + s > 0);
              mma_commit(kpempty + 8 * (subs & 1));
            }
            if (!ok) break;
            mma_commit(kvfull);
            ++kvs;
            mma_commit(empty + 8 * kValue);
          } else {
            bar_arrive(empty + 8 * kValue);
          }
        }
        bar_arrive(gempty + 8 * (gs));
      }
      mma_commit(alldone + 8 * (1));
      drain(alldone + 8 * (1), 1);
    }
  } else if (warp == 2) {
    // ---- gates ----
    Walker w;
    w.seek(&plan, nch, range.u0);
    for (int64_t i = 0; i < count; ++i) {
      const int unit = static_cast<int>(i);
      const int gs = unit % kGateStages, n = w.rows(), row0 = w.row0();
      const int hv = w.ht / plan.tiles;
      float g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        g[j] = 4 * lane + j < n ? kLog2e * p.g.at(row0 + 4 * lane + j, hv) : 0.f;
      if (unit >= kGateStages && !(ok = CATTN_WARP_WAIT(gempty + 8 * (gs), unit / kGateStages - 1))) break;
      Gate& gt = gates[gs];
      make_gate(gt, g, lane);
      if (lane == 0) {
        gt.row0 = row0;
        gt.n = n;
        gt.ht = w.ht;
        gt.seq = w.seq;
        int f = 0;
        const bool first = w.first();
        if (i == 0 || first) f |= kSegment;
        if ((f & kSegment) && !first) f |= kMiddle;
        if (!first || p.initial) f |= kHasState;
        if (w.last() && p.fin) f |= kFinish;
        if ((!w.last() && i + 1 < count) || (f & kFinish)) f |= kNeedKv;
        if (range.u0 + i >= tail.u0 && tail.closed) f |= kSplitSeq;
        gt.flags = f;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gfull + 8 * (gs));
      if (i + 1 < count) w.next();
    }
  }
  } else if (warp < 8) {
    // ---- scores to P, and the outputs ----
    const int wq = warp - 4, row = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    int scs = 0;
    for (int unit = 0; unit < count; ++unit) {
      const int gs = unit % kGateStages;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * (gs), unit / kGateStages))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, row0 = gt.row0, ht = gt.ht;
      const bool inter = gt.flags & kHasState;
      const float er = gt.er[row];
      if (n > 0) {
        const float lp = gt.lp[row];
        if (!(ok = CATTN_WARP_WAIT(scfull, scs))) break;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < (FINE ? kFineTokens / 32 : 4); ++b) {
          uint32_t x[32], y[16];
          const auto put = [&](int i, f2 v) {  // one term is rounded at once: 110 us against 114
            if (FINE)
              put_pair(x, i, v);
            else
              y[i] = f2_to_bf16x2(v);
          };
          if (b <= wq) {
            tmem_ld32(tmem + lanes + b * 32, x);
            tmem_wait_ld();
            tmem_use32(x);
          }
          if (b < wq) {
            float e = lp;
#pragma unroll 1
            for (int i = b + 1; i < wq; ++i) e += gt.block[i];
            const f2 ut = f2_splat(exp2_fast(e));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const ulonglong2 ws = *reinterpret_cast<const ulonglong2*>(&gt.ws[b * 32 + i * 4]);
              put(2 * i, f2_mul(pair(x, 2 * i), f2_mul(ut, ws.x)));
              put(2 * i + 1, f2_mul(pair(x, 2 * i + 1), f2_mul(ut, ws.y)));
            }
          } else if (b == wq) {
            // the diagonal block: the decay from s to t as a running product down from t
            float w = 1.f;
#pragma unroll
            for (int i = 7; i >= 0; --i) {
              const float4 a = *reinterpret_cast<const float4*>(&gt.a[b * 32 + 4 * i]);
              float v[4];
#pragma unroll
              for (int j = 3; j >= 0; --j) {
                const int c = 4 * i + j;
                v[j] = c <= lane ? __uint_as_float(x[c]) * w : 0.f;
                if (c <= lane) w *= j == 3 ? a.w : j == 2 ? a.z : j == 1 ? a.y : a.x;
              }
              put(2 * i, f2_pack(v[0], v[1]));
              put(2 * i + 1, f2_pack(v[2], v[3]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) put(i, 0);
          }
          if (FINE)
            put_p<FINE>(tmem + lanes, b, x);
          else
            tmem_st16(tmem + lanes + b * 16, y);
        }
        tmem_wait_st();
        tc_fence_before();
        if (!(ok = CATTN_WARP_WAIT(full + 8 * kValue, scs))) break;
        if (n < kChunk) {
          zero_rows(smem + kValue * kTileBytes, p.V - ht % plan.tiles * 128 > kPanelCols ? 2 : 1, n, row,
                    128);
          cconv::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) {
          bar_arrive(pfull);
          if (n < kChunk) bar_arrive(vfixed);
        }
        if (!(ok = CATTN_WARP_WAIT(ofull, scs))) break;
        ++scs;
        tc_fence_after();
        const int vt = ht % plan.tiles, vw = min(128, p.V - vt * 128);
        uint16_t* dst = p.o + (static_cast<int64_t>(row0 + row) * p.Hv + ht / plan.tiles) * p.V +
                        vt * 128;
        const f2 es = f2_splat(p.scale * er), sc = f2_splat(p.scale);
        // The outputs of a full chunk leave through the buffer of the bf16 state (Q S is done, and
        // the next state waits for `stored`) by TMA: a row a thread of plain stores kept the load /
        // store unit, and every other role, busy for some 2000 cycles a chunk.
        const bool whole = n == kChunk;
#pragma unroll 1
        for (int c = 0; c < vw; c += 32) {
          uint32_t x[32], z[32];
          tmem_ld32(tmem + lanes + 128 + c, x);
          if (inter) {
            tmem_ld32(tmem + lanes + 256 + c, z);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0;
          }
          tmem_wait_ld();
          tmem_use32(x);
          tmem_use32(z);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = f2_to_bf16x2(f2_fma(es, pair(z, i), f2_mul(sc, pair(x, i))));
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sts128(smem + kOffS + (c >> 6) * kPanelBytes + swizzled(row, ((c >> 3) & 7) + i), x[4 * i],
                     x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          } else if (row < n) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + 8 * i < vw)
                *reinterpret_cast<uint4*>(dst + c + 8 * i) =
                    make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
        tc_fence_before();
        if (whole) cconv::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(ofree), bar_arrive(osync);
        if (!(ok = CATTN_WARP_WAIT(osync, scs - 1))) break;  // the four warps' rows are staged
        if (row == 0) {
          if (whole) {
#pragma unroll 1
            for (int c = 0; c < vw; c += kPanelCols)
              store_box(&p.mo, smem + kOffS + (c >> 6) * kPanelBytes, vt * 128 + c, ht / plan.tiles,
                        row0);
            stores_commit();
            stores_wait_read();
          }
          set_count(stored, scs);
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * (gs));
    }
  } else if (warp < 12) {
    // ---- decayed keys ----
    set_registers<104, false>();
    const int kt = threadIdx.x - (12 - kKeyWarps) * 32;
    int chunk = 0, subs = 0;
    for (int unit = 0; unit < count && ok; ++unit) {
      const int gs = unit % kGateStages;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * (gs), unit / kGateStages))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n;
      if (n > 0) {
        const int key = chunk & 1;
        if (!(ok = CATTN_WARP_WAIT(full + 8 * key, chunk >> 1))) break;
        ++chunk;
        if (gt.flags & kNeedKv) {
          const uint32_t src = smem + key * kTileBytes;
          const int blocks = (n + kSub - 1) / kSub;
#pragma unroll 1
          for (int b = 0; b < blocks; ++b, ++subs) {
            if (subs >= 2 && !(ok = CATTN_WARP_WAIT(kpempty + 8 * (subs & 1), (subs >> 1) - 1))) break;
            const uint32_t dst = smem + kOffKp + (subs & 1) * kSubBytes;
#pragma unroll 2
            for (int e = kt; e < kSub * 8 * pk; e += kKeyWarps * 32) {
              const int r = e >> (2 + pk), piece = e & (8 * pk - 1), t = b * kSub + r;
              const uint32_t q = piece >> 3, at = swizzled(r, piece & 7);
              // (rows b * kSub + r and r have the same place in their groups of 8)
              uint4 in = lds128_at(src + q * kPanelBytes + b * kSub * 128 + at);
              if (t >= n) in = make_uint4(0, 0, 0, 0);
              store_split(in, gt.kw[t], dst + q * kSubPanel + at, kSubTile);
            }
            cconv::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(kpfull + 8 * (subs & 1));
          }
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(empty + 8 * key);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * (gs));
    }
  } else {
    // ---- the state: a row of 128 columns a thread ----
    set_registers<208, true>();
    const int krow = threadIdx.x - 384;
    const uint32_t lanes = static_cast<uint32_t>(krow & ~31) << 16;
    f2 S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0;
    int kvs = 0, pubs = 0, done = 0;  // done: chunks with outputs before this one
    for (int unit = 0; unit < count && ok; ++unit) {
      const int gs = unit % kGateStages;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * (gs), unit / kGateStages))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, flags = gt.flags, ht = gt.ht;
      const int hv = ht / plan.tiles, vt = ht % plan.tiles;
      const int vw = min(128, p.V - vt * 128);
      if (flags & kSegment) {
        const int64_t slot = p.slots.of(gt.seq);
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0;
        if (flags & kMiddle) {
          // what the ranges before this one hand on, back to the one where the sequence began
          gather_state(S, p.carry, p.decay, blockIdx.x, parts, -1, p.joined, krow);
        } else if (p.initial && slot >= 0 && krow < p.K) {
          const float* src = p.initial + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128;
          const ulonglong2* from = reinterpret_cast<const ulonglong2*>(
              p.copy + static_cast<int64_t>(blockIdx.x) * kStateFloats);
          const bool saved = (flags & kSplitSeq) && p.fin;  // final_state may have replaced it
          if (saved) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const ulonglong2 x = from[i * 128 + krow];
              S[2 * i] = x.x, S[2 * i + 1] = x.y;
            }
          } else {
            load_state(S, src, vw);
          }
        }
      }
      if (n > 0 && (flags & kHasState)) {
        if (pubs > 0 && !(ok = CATTN_WARP_WAIT(sempty, pubs - 1))) break;
        if (!(ok = __all_sync(0xffffffffu, wait_count(stored, done)))) break;
        ++pubs;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sts128(smem + kOffS + i / 8 * kPanelBytes + swizzled(krow, i % 8),
                 f2_to_bf16x2(S[4 * i]), f2_to_bf16x2(S[4 * i + 1]), f2_to_bf16x2(S[4 * i + 2]),
                 f2_to_bf16x2(S[4 * i + 3]));
        cconv::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(sfull);
      }
      if (n > 0 && (flags & kNeedKv)) {
        const f2 d = f2_splat(gt.total);
        if (!(ok = CATTN_WARP_WAIT(kvfull, kvs))) break;
        ++kvs;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32];
          tmem_ld32(tmem + lanes + 384 + c * 32, x);
          tmem_wait_ld();
          tmem_use32(x);
#pragma unroll
          for (int i = 0; i < 16; ++i) S[c * 16 + i] = f2_fma(d, S[c * 16 + i], pair(x, i));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(kvfree);
      }
      if (n > 0) ++done;
      if ((flags & kFinish) && krow < p.K &&
          (!plan.idx || (plan.small ? small.usable != 0 : plan.status[0] == CCONV_OK))) {
        const int64_t slot = p.slots.of(gt.seq);
        float* dst = p.fin + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128;
        if (slot >= 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (8 * i < vw) st_pairs(dst + 8 * i, &S[4 * i]);
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * (gs));
    }
  }
  }
  if (threadIdx.x == 128) stores_wait();  // the thread that stored: all of it is written
  if (!ok) atomicOr(&g_fault_fwd, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// ----------------------------------------------------------------------------------------
// the states that ranges hand on
// ----------------------------------------------------------------------------------------
// The state at the end of a range is one sum over its tail's tokens with the decay from each to
// the end (REV: to the start), so all chunks accumulate in one TMEM tile and nothing is read
// until it is whole.  The chunks are taken from that end on: once the decay has run out of
// fp32 (2^-127), the rest would add zeros and is not read.  The keys' first terms and their
// small ones accumulate apart: the tensor cores' sums are cut off, not rounded, at each step,
// and in one tile the small terms' steps tripled that error (1.8e-6 of the final states of 16
// sequences of 16384 rows in all, against 1e-6).
constexpr int kTailKeyWarps = 16;
constexpr int kTailThreads = (4 + kTailKeyWarps) * 32;
constexpr int kTailSlots = 4;   // two chunks of two tiles
constexpr int kTailBlocks = 3;
constexpr int kTailGates = 3;
struct alignas(16) TailGate {
  float w[kChunk];
  int row0, n, ht, seq, last;
};
constexpr int kTailKp = kTailSlots * kTileBytes;
constexpr int kTailOffGates = kTailKp + kTailBlocks * kSubBytes;
constexpr int kTailBars = kTailOffGates + kTailGates * sizeof(TailGate);
constexpr int kTailBytes = kTailBars + 32 * 8 + 1024;
static_assert(kTailBytes <= 232448, "shared memory of one CTA");

template <bool REV>
__device__ __forceinline__ void tail_state(const ChunkArgs& p, uint8_t* raw, SmallPlan& small) {
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  TailGate* gates = reinterpret_cast<TailGate*>(base + kTailOffGates);
  const uint32_t smem = smem_addr(base);
  const uint32_t full = smem + kTailBars, empty = full + 8 * kTailSlots;
  const uint32_t gfull = empty + 8 * kTailSlots, gempty = gfull + 8 * kTailGates;
  const uint32_t kpfull = gempty + 8 * kTailGates, kpempty = kpfull + 8 * kTailBlocks;
  const uint32_t vfixed = kpempty + 8 * kTailBlocks, alldone = vfixed + 8;
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(base + kTailBars + 31 * 8);
  float* passed = reinterpret_cast<float*>(tmem_at + 1);  // log2 of the tail's decay

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTailSlots; ++i) {
      bar_init(full + 8 * i, 1);
      bar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kTailGates; ++i) {
      bar_init(gfull + 8 * i, 1);
      bar_init(gempty + 8 * i, kTailKeyWarps + 2);
    }
    for (int i = 0; i < kTailBlocks; ++i) {
      bar_init(kpfull + 8 * i, kTailKeyWarps);
      bar_init(kpempty + 8 * i, 1);
    }
    bar_init(vfixed, kTailKeyWarps);
    bar_init(alldone, 1);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_at, 256);
  if (warp == 0 && lane == 0 && p.rows > 0) {
    cconv::prefetch_tensormap(&p.mk);
    cconv::prefetch_tensormap(&p.mv);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  Plan plan = p.plan;
  if (plan.small) small_plan(plan, small, p.report && blockIdx.x == 0, &g_fault_fwd);

  int nch;
  const int64_t units = unit_count(plan, nch);
  const int64_t parts = range_count(plan, gridDim.x, units);
  const int place = blockIdx.x / plan.group, member = blockIdx.x % plan.group;
  Range range{0, 0};
  if (place < parts) range = range_of(units, parts, place);
  const Tail tail = tail_of<REV>(plan, nch, units, range);
  const int count = static_cast<int>(tail.u1 - tail.u0);
  const int64_t start = REV ? tail.u0 : tail.u1 - 1;
  const int pk = p.K > kPanelCols ? 2 : 1;
  bool ok = true;  // no wait of this thread's has given up
  if (count == 0 && threadIdx.x == 0) p.decay[blockIdx.x] = kNoTail;
  if (count > 0) {
    if (warp == 0) {
      // ---- tiles: as the gates ask for them ----
      if (elect_one()) {
        int tile = 0;
        for (int unit = 0; unit < count && ok; ++unit) {
          const int gs = unit % kTailGates;
          if (!(ok = CATTN_WAIT(gfull + 8 * gs, unit / kTailGates))) break;
          const TailGate& gt = gates[gs];
          const int hv = gt.ht / plan.tiles, vt = gt.ht % plan.tiles, row = gt.row0;
          const int pv = p.V - vt * 128 > kPanelCols ? 2 : 1;
          const bool last = gt.last;
#pragma unroll 1
          for (int j = 0; j < 2 && ok; ++j, ++tile) {
            const int slot = tile % kTailSlots, use = tile / kTailSlots;
            if (use > 0 && !(ok = CATTN_WAIT(empty + 8 * slot, use - 1))) break;
            const int panels = j ? pv : pk;
            bar_expect(full + 8 * slot, panels * kPanelBytes);
#pragma unroll 1
            for (int c = 0; c < panels; ++c)
              load_box(smem + slot * kTileBytes + c * kPanelBytes, j ? &p.mv : &p.mk, full + 8 * slot,
                       (j ? vt * 128 : 0) + c * kPanelCols, j ? hv : hv / p.ratio, row);
          }
          bar_arrive(gempty + 8 * gs);
          if (last) break;
        }
        for (int i = 0; i < kTailSlots; ++i)
          drain(full + 8 * i, (tile + kTailSlots - 1 - i) / kTailSlots);
      }
    } else if (warp == 1) {
      // ---- matrix products ----
      if (elect_one()) {
        int subs = 0;
        for (int unit = 0; unit < count && ok; ++unit) {
          const int gs = unit % kTailGates;
          if (!(ok = CATTN_WAIT(gfull + 8 * gs, unit / kTailGates))) break;
          const TailGate& gt = gates[gs];
          const int n = gt.n;
          const bool last = gt.last;
          const int nv = (min(128, p.V - gt.ht % plan.tiles * 128) + 15) / 16 * 16;
          const int tk = 2 * unit, tv = tk + 1;
          if (!(ok = CATTN_WAIT(full + 8 * (tv % kTailSlots), tv / kTailSlots))) break;
          if (n < kChunk && !(ok = CATTN_WAIT(vfixed, 0))) break;
          const uint32_t d = mma_desc(nv, true, true);
          const int blocks = (n + kSub - 1) / kSub;
#pragma unroll 1
          for (int b = 0; b < blocks; ++b, ++subs) {
            const int kb = subs % kTailBlocks;
            if (!(ok = CATTN_WAIT(kpfull + 8 * kb, subs / kTailBlocks))) break;
            tc_fence_after();
            const uint64_t da = tile_desc(smem + kTailKp + kb * kSubBytes, kSubPanel);
            const uint64_t db = tile_desc(smem + tv % kTailSlots * kTileBytes + b * kSub * 128, kPanelBytes);
#pragma unroll
            for (int s = 0; s < 2 * kSplit; ++s)  // term s / 2, tokens [16 (s & 1), + 16)
              mma_ss(tmem + (s < 2 ? 0 : 128), da + (s >> 1) * (kSubTile / 16) + (s & 1) * kRowStep,
                     db + (s & 1) * kRowStep, d, subs > 0 || (s != 0 && s != 2));
            mma_commit(kpempty + 8 * kb);
          }
          if (!ok) break;
          // (the keys' tile was read before its last block was handed over)
          mma_commit(empty + 8 * (tk % kTailSlots));
          mma_commit(empty + 8 * (tv % kTailSlots));
          bar_arrive(gempty + 8 * gs);
          if (last) break;
        }
        mma_commit(alldone);
        drain(alldone, 1);
      }
    } else if (warp == 2) {
      // ---- gates ----
      Walker w;
      w.seek(&plan, nch, start, member);
      float g[4], run = 0.f;
      const int hv = w.ht / plan.tiles;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        g[j] = 4 * lane + j < w.rows() ? kLog2e * p.g.at(w.row0() + 4 * lane + j, hv) : 0.f;
      for (int unit = 0; unit < count; ++unit) {
        const int gs = unit % kTailGates, n = w.rows(), row0 = w.row0();
        if (unit >= kTailGates && !(ok = CATTN_WARP_WAIT(gempty + 8 * gs, unit / kTailGates - 1))) break;
        TailGate& gt = gates[gs];
        // sums over the tokens after (REV: before) each of this lane's four, in the chunk
        const float own = (g[0] + g[1]) + (g[2] + g[3]);
        float sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float x = REV ? __shfl_up_sync(0xffffffffu, sum, o) : __shfl_down_sync(0xffffffffu, sum, o);
          if (REV ? lane >= o : lane + o < 32) sum += x;
        }
        const float all = __shfl_sync(0xffffffffu, sum, REV ? 31 : 0);
        const float next = REV ? __shfl_up_sync(0xffffffffu, sum, 1) : __shfl_down_sync(0xffffffffu, sum, 1);
        float e = run + (lane == (REV ? 0 : 31) ? 0.f : next);
        float v[4];
        if (REV) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = exp2_fast(e += g[j]);
        } else {
#pragma unroll
          for (int j = 3; j >= 0; --j) {
            v[j] = exp2_fast(e);
            e += g[j];
          }
        }
        *reinterpret_cast<float4*>(&gt.w[4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
        run += all;
        const bool last = unit + 1 == count || run < -127.f;
        if (lane == 0) {
          gt.row0 = row0;
          gt.n = n;
          gt.ht = w.ht;
          gt.seq = w.seq;
          gt.last = last;
          if (last) *passed = unit + 1 == count ? run : -INFINITY;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(gfull + 8 * gs);
        if (last) break;
        w.step<!REV>();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          g[j] = 4 * lane + j < w.rows() ? kLog2e * p.g.at(w.row0() + 4 * lane + j, hv) : 0.f;
      }
    } else if (warp >= 4) {
      // ---- decayed keys ----
      const int kt = threadIdx.x - 128;
      int subs = 0, ht = 0, seq = 0;
      for (int unit = 0; unit < count && ok; ++unit) {
        const int gs = unit % kTailGates;
        if (!(ok = CATTN_WARP_WAIT(gfull + 8 * gs, unit / kTailGates))) break;
        const TailGate& gt = gates[gs];
        const int n = gt.n, tk = 2 * unit, tv = tk + 1;
        const bool last = gt.last;
        ht = gt.ht;
        seq = gt.seq;
        if (n < kChunk) {  // a sequence's last chunk: once in a tail
          if (!(ok = CATTN_WARP_WAIT(full + 8 * (tv % kTailSlots), tv / kTailSlots))) break;
          zero_rows(smem + tv % kTailSlots * kTileBytes,
                    p.V - ht % plan.tiles * 128 > kPanelCols ? 2 : 1, n, kt, kTailKeyWarps * 32);
          cconv::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive(vfixed);
        }
        if (!(ok = CATTN_WARP_WAIT(full + 8 * (tk % kTailSlots), tk / kTailSlots))) break;
        const uint32_t src = smem + tk % kTailSlots * kTileBytes;
        const int blocks = (n + kSub - 1) / kSub;
        const int r = kt >> (2 + pk), piece = kt & (8 * pk - 1);
        const uint32_t q = piece >> 3, at = swizzled(r, piece & 7);
#pragma unroll 1
        for (int b = 0; b < blocks; ++b, ++subs) {
          const int kb = subs % kTailBlocks, t = b * kSub + r;
          if (subs >= kTailBlocks && !(ok = CATTN_WARP_WAIT(kpempty + 8 * kb, subs / kTailBlocks - 1)))
            break;
          if (r < kSub) {
            uint4 in = lds128_at(src + q * kPanelBytes + b * kSub * 128 + at);
            if (t >= n) in = make_uint4(0, 0, 0, 0);
            store_split(in, gt.w[t], smem + kTailKp + kb * kSubBytes + q * kSubPanel + at, kSubTile);
            cconv::fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) bar_arrive(kpfull + 8 * kb);
        }
        if (!ok) break;
        if (lane == 0) bar_arrive(gempty + 8 * gs);
        if (last) break;
      }
      if (warp < 8 && ok && (ok = CATTN_WARP_WAIT(alldone, 0))) {
        tc_fence_after();
        const int krow = threadIdx.x - 128;
        const uint32_t lanes = static_cast<uint32_t>(krow & ~31) << 16;
        const int hv = ht / plan.tiles, vt = ht % plan.tiles, vw = min(128, p.V - vt * 128);
        const int64_t slot = p.slots.of(seq);
        const float rest = exp2_fast(*passed);
        const bool start_state = !REV && tail.closed && p.initial && slot >= 0 && krow < p.K;
        const float* src = p.initial + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128;
        float4* to = reinterpret_cast<float4*>(p.carry + static_cast<int64_t>(blockIdx.x) * kStateFloats);
        // (the outputs' kernel reads this copy: by then final_state may have replaced the state)
        float4* copy = reinterpret_cast<float4*>(p.copy + static_cast<int64_t>(blockIdx.x) * kStateFloats);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32], y[32];
          tmem_ld32(tmem + lanes + c * 32, x);
          tmem_ld32(tmem + lanes + 128 + c * 32, y);
          tmem_wait_ld();
          tmem_use32(x);
          tmem_use32(y);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f);
            if (start_state && c * 32 + 4 * i < vw)
              s0 = *reinterpret_cast<const float4*>(src + c * 32 + 4 * i);
            to[(c * 8 + i) * 128 + krow] =
                make_float4(fmaf(rest, s0.x, __uint_as_float(x[4 * i])),
                            fmaf(rest, s0.y, __uint_as_float(x[4 * i + 1])),
                            fmaf(rest, s0.z, __uint_as_float(x[4 * i + 2])),
                            fmaf(rest, s0.w, __uint_as_float(x[4 * i + 3])));
            if (!REV && tail.closed && p.initial && p.fin) copy[(c * 8 + i) * 128 + krow] = s0;
          }
        }
        if (krow == 0) p.decay[blockIdx.x] = tail.closed ? kChainStart : rest;
      }
    }
  }
  if (!ok) atomicOr(&g_fault_fwd, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 256);
  }
}

__global__ void __launch_bounds__(kTailThreads, 1)
    cattn_linear_tail_kernel(const __grid_constant__ ChunkArgs p) {
  extern __shared__ uint8_t raw[];
  __shared__ SmallPlan small;
  tail_state<false>(p, raw, small);
}
// The backward's: the states and their gradients (blockIdx.y = 1) in one launch.  How much a range
// has to read depends on its gates, and the CTAs that are done early make room for others: 67 us
// against 72 for two launches (16384 rows, 16 heads), 4 of 62 us of a small ragged call.  (The
// forward has a kernel of its own: in this one it took 2 us longer.)
__global__ void __launch_bounds__(kTailThreads, 1)
    cattn_linear_tails_kernel(const __grid_constant__ ChunkArgs states, const __grid_constant__ ChunkArgs grads) {
  extern __shared__ uint8_t raw[];
  __shared__ SmallPlan small;
  if (blockIdx.y == 0)
    tail_state<false>(states, raw, small);
  else
    tail_state<true>(grads, raw, small);
}

// Joins what the ranges hand on along each chain of ranges of one sequence, in place: carry[i]
// becomes the whole state at the end (REV: start) of CTA i's range.  For long chains: a sweep's CTA
// would read every state of its chain, one after the other (0.8 us each); here each thread follows 16 bytes of it along the chain with kScanAhead reads in
// flight.  grid: (ranges, slices of a state, directions); the CTAs of ranges that do not start a
// chain have nothing to do.
constexpr int kScanThreads = 256, kScanAhead = 8, kMaxRanges = 1024;
constexpr int kScanSlices = kStateFloats / 4 / kScanThreads;
struct ScanArgs {
  float* carry[2];
  const float* decay[2];
  int grid, group;
};
__global__ void __launch_bounds__(kScanThreads) cattn_linear_scan_kernel(const __grid_constant__ ScanArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float decay[kMaxRanges];
  const int rev = blockIdx.z, by = rev ? -p.group : p.group, first = blockIdx.x;
  for (int i = threadIdx.x; i < p.grid; i += kScanThreads) decay[i] = p.decay[rev][i];
  __syncthreads();
  if (decay[first] != kChainStart) return;
  constexpr int64_t kPitch = kStateFloats / 4;
  float4* states = reinterpret_cast<float4*>(p.carry[rev]) + blockIdx.y * kScanThreads + threadIdx.x;
  float4 run = states[first * kPitch];
  for (int i = first + by;;) {
    int n = 0;  // the next ranges that go on with the chain
    float4 x[kScanAhead];
#pragma unroll
    for (int j = 0; j < kScanAhead; ++j) {
      const int r = i + j * by;
      // (a NaN decay goes on with the chain: all that follows it is NaN)
      if (n == j && r >= 0 && r < p.grid && decay[r] != kChainStart && decay[r] != kNoTail) {
        x[j] = states[r * kPitch];
        n = j + 1;
      }
    }
#pragma unroll
    for (int j = 0; j < kScanAhead; ++j)
      if (j < n) {
        const float d = decay[i + j * by];
        run.x = fmaf(d, run.x, x[j].x);
        run.y = fmaf(d, run.y, x[j].y);
        run.z = fmaf(d, run.z, x[j].z);
        run.w = fmaf(d, run.w, x[j].w);
        states[(i + j * by) * kPitch] = run;
      }
    if (n < kScanAhead) return;
    i += n * by;
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

// Map of a [total, H, C] tensor read in boxes of `cols` channels (64, or 32) of one head and `tokens` tokens.
int encode_tile_map(CUtensorMap* map, const Rows& x, int64_t total, int64_t H, int64_t C, int tokens, int cols) {
  auto enc = encode_fn();
  if (!enc) return CCONV_ERR_CUDA;
  // strides over dimensions of extent 1 are the caller's to leave unset
  const int64_t sh = H > 1 ? x.sh : C, st = total > 1 ? x.st : C * H;
  cuuint64_t dims[3] = {(cuuint64_t)C, (cuuint64_t)H, (cuuint64_t)total};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2u, (cuuint64_t)st * 2u};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(cols), 1u, static_cast<cuuint32_t>(tokens)};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(x.p), dims, strides, box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, cols == kPanelCols ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CCONV_OK : CCONV_ERR_CUDA;
}

// Map of the [parts, total, C] fp32 sums, written in boxes of 32 channels of one part and 128
// tokens.
int encode_part_map(CUtensorMap* map, float* x, int64_t total, int64_t parts, int64_t C) {
  auto enc = encode_fn();
  if (!enc) return CCONV_ERR_CUDA;
  cuuint64_t dims[3] = {(cuuint64_t)C, (cuuint64_t)parts, (cuuint64_t)total};
  cuuint64_t strides[2] = {(cuuint64_t)(total * C) * 4u, (cuuint64_t)C * 4u};
  cuuint32_t box[3] = {32u, 1u, kChunk};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, x, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? CCONV_OK : CCONV_ERR_CUDA;
}

// A chain has at most ceil(ranges / (heads * tiles)) + 1 states.  With 10 of them at most (16 heads)
// the scan's launch costs more than it saves (forward of 16384 rows 112 us against 108); with 31
// (4 heads) it saves a third of a backward (62 us against 102).
constexpr int kLongChain = 12;
int launch_scan(const ChunkCall& c, float* forward, float* backward, bool* scanned, cudaStream_t stream) {
  const int tiles = (c.s.V + 127) / 128;
  *scanned = c.grid > kLongChain * c.s.Hv * tiles && c.grid <= kMaxRanges;
  if (!*scanned) return CCONV_OK;
  ScanArgs a{};
  a.carry[0] = forward, a.carry[1] = backward;
  const int64_t decays = static_cast<int64_t>(c.grid) * 2 * kStateFloats;
  a.decay[0] = forward + decays, a.decay[1] = backward ? backward + decays : nullptr;
  a.grid = c.grid, a.group = c.group;
  return launch_pdl(cattn_linear_scan_kernel, dim3(c.grid, kScanSlices, backward ? 2 : 1),
                    dim3(kScanThreads), 0, stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

static int chunk_args(const ChunkCall& c, ChunkArgs& a) {
  int rc = CCONV_OK;
  if (c.s.total > 0) {
    rc = bind_context();
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K);
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K);
    if (rc == CCONV_OK) rc = encode_tile_map(&a.mv, c.v, c.s.total, c.s.Hv, c.s.V);
    if (rc == CCONV_OK && c.o)
      rc = encode_tile_map(&a.mo, Rows{c.o, int64_t(c.s.Hv) * c.s.V, c.s.V}, c.s.total, c.s.Hv, c.s.V);
    if (rc != CCONV_OK) return rc;
  }
  const int tiles = (c.s.V + 127) / 128;
  a.plan = Plan{c.cu, c.cstart, c.s.nseq, tiles, c.s.Hv, c.group, c.cstart == nullptr, c.s.total,
                c.slots.idx, c.slots.S, c.status};
  a.g = c.g;
  a.slots = c.slots;
  a.initial = c.initial;
  a.fin = c.fin;
  a.report = c.o == nullptr;
  a.o = c.o;
  a.carry = c.carry;
  a.copy = c.carry + static_cast<int64_t>(c.grid) * kStateFloats;
  a.decay = a.copy + static_cast<int64_t>(c.grid) * kStateFloats;
  a.scale = c.scale;
  a.rows = c.s.total;
  a.ratio = c.s.Hv / c.s.Hk;
  a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  return CCONV_OK;
}

template <class... Args>
static int launch(void (*kern)(Args...), dim3 grid, int threads, int bytes, cudaStream_t stream,
                  const Args&... args) {
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), bytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(kern, grid, dim3(threads), bytes, stream, args...) == cudaSuccess ? CCONV_OK
                                                                                     : CCONV_ERR_CUDA;
}

int launch_chunk_states(const ChunkCall& states, const ChunkCall& grads, cudaStream_t stream) {
  ChunkArgs a{}, b{};
  int rc = chunk_args(states, a);
  if (rc == CCONV_OK) rc = chunk_args(grads, b);
  if (rc != CCONV_OK) return rc;
  return launch(cattn_linear_tails_kernel, dim3(states.grid, 2), kTailThreads, kTailBytes, stream, a, b);
}

int launch_chunk_fwd(const ChunkCall& c, cudaStream_t stream) {
  ChunkArgs a{};
  int rc = chunk_args(c, a);
  // with at most 128 rows no sequence has a second chunk, and nothing is handed on
  if (rc == CCONV_OK && c.s.total > kChunk) {
    rc = launch(cattn_linear_tail_kernel, dim3(c.grid), kTailThreads, kTailBytes, stream, a);
    bool joined = false;
    if (rc == CCONV_OK) rc = launch_scan(c, c.carry, nullptr, &joined, stream);
    a.joined = joined;
  }
  if (rc != CCONV_OK) return rc;
  return launch(c.s.total <= kFineTokens ? cattn_linear_chunk_kernel<true> : cattn_linear_chunk_kernel<false>,
                dim3(c.grid), kFwdThreads, kFwdBytes, stream, a);
}

size_t chunk_fwd_bytes(int grid) {
  return static_cast<size_t>(grid) * (2 * kStateFloats + 4) * sizeof(float);
}

}  // namespace cattn
