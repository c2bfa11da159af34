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
// three bf16 terms (24 bits; with two, the 16 bits showed: 1e-6 to 7e-6 of dg, where an initial state
// meets a few tokens).  There is room for two terms at a time: the first replaces the second once
// that is read (8 % of the time).  Each range also gives dg at its start as the product of the two
// whole fp32 states, and the sums in between are tied to these anchors.
//
// Roles of the 20 warps: one warp streams tiles, one thread issues the products of the outputs
// and one those of the state, one warp makes the gates; four warps each turn score tiles into P,
// make decayed rows, keep the state, and finish the outputs.  The ring's four slots hold one
// tile each of v, do, k and q, refilled as soon as its last reader is done.  TMEM:
//   KV = false  [0,128) M1, then P   [128,256) M2   [256,384) dq   [384,512) K^T V
//   KV = true   [0,128) M1, then P1 | Q^T dO (columns 0-63)   [128,256) M2, then P2 | Q^T dO (64-)
//               [256,384) dk         [384,512) dv
// The products with the state are scaled in place by their rows' decays, and P's products
// accumulate on them.  Finished tiles leave by TMA through the buffer of the bf16 state, as the
// forward's outputs do.
//
// Shared memory: the tensor cores read both operands of every product there (64 cycles
// of 128 bytes for 128 x 128 x 16), some 5500 cycles a chunk, and the warps' accesses and TMEM
// loads add as much again.  Bound by the chain of the roles, 17000 (dq) and 20000 cycles a chunk, as
// there is no room for a second slot a tile or, in TMEM, for D's product beside the scores (tensor
// cores active 23 % of the time, load / store unit 31 to 37 %, DRAM 23 %).  16384 rows in 2
// sequences, 16 value heads on 8 key heads of 128: 135 and 171 us of the backward's 385.  The
// compiler spills some 150 (dq) to 190 bytes a thread of the roles that share these kernels.
#include "attn_chunk.cuh"
#include "attn_chunk_host.h"

#include <atomic>

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

constexpr int kBwdThreads = 640;
constexpr int kBwdGates = 2;
constexpr int kBwdReaders = 4 * 4 + 2;            // warps and threads that read a gate
constexpr int kBlock = 16;                        // tokens of one decayed block
constexpr int kBlockPanel = kBlock * 128;
constexpr int kBlockTile = 2 * kBlockPanel;
constexpr int kBlockBytes = kSplit * kBlockTile;
enum Slot : int { kV = 0, kDo = 1, kK = 2, kQ = 3, kBwdSlots = 4 };

// shared memory, from a 1024-byte boundary
constexpr int kOffKp = kBwdSlots * kTileBytes;          // two blocks of decayed rows
constexpr int kOffS = kOffKp + 2 * kBlockBytes;         // two bf16 terms of the state; outputs
constexpr int kOffGates = kOffS + 2 * kTileBytes;
constexpr int kOffBars = kOffGates + kBwdGates * sizeof(Gate);
constexpr int kOffCounts = kOffBars + 40 * 8;           // [4 warps][kMaxGroup]: see ring_tile
constexpr int kMaxGroup = 8;
constexpr int kBwdBytes = kOffCounts + 4 * kMaxGroup * 4 + 1024;
static_assert(kBwdBytes <= 232448, "shared memory of one CTA");

struct BwdArgs {
  CUtensorMap mq, mk, mv, mo;
  CUtensorMap out_k, out_v;  // dq or dk (or their parts) and dv
  Plan plan;
  Gates g;
  Slots slots;
  const float* initial;
  float* dinit;             // KV: [nseq, Hv, K, V] or NULL
  uint16_t *dqk, *dv;       // dq or dk in bf16 where one unit makes a row of them, else
  float* part;              // [units' (head, tile)][total][K] partial sums, or
  float4* ring;             // [grid][2][K / 4][128]: two chunks' partial sums of each CTA
  float* dots;              // [2][heads * tiles][total]
  float* states;            // [grid] the states before the ranges: the first sweep's, for anchors
  float* anchors;           // KV: [grid][4] parts of scale <D, S> there
  const float* carry;       // states handed on
  const float* decay;
  float scale;
  int rows, ratio, Hk, Hv, K, V;
  int joined;               // the states handed on are whole
};

#define CATTN_WAIT(bar, parity) (wait_phase((bar), static_cast<uint32_t>(parity) & 1u))
#define CATTN_WARP_WAIT(bar, parity) (__all_sync(0xffffffffu, CATTN_WAIT(bar, parity)))

// Dot of 32 fp32 values with columns [c, c + 32) of row `row` of a bf16 tile.
__device__ __forceinline__ f2 dot_tile(uint32_t tile, int row, int c, const uint32_t* x, f2 dot) {
  const uint32_t at = tile + (c >> 6) * kPanelBytes;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = lds128_at(at + swizzled(row, ((c >> 3) & 7) + i));
    dot = f2_fma(bf16x2_to_f2(w.x), pair(x, 4 * i), dot);
    dot = f2_fma(bf16x2_to_f2(w.y), pair(x, 4 * i + 1), dot);
    dot = f2_fma(bf16x2_to_f2(w.z), pair(x, 4 * i + 2), dot);
    dot = f2_fma(bf16x2_to_f2(w.w), pair(x, 4 * i + 3), dot);
  }
  return dot;
}

__device__ __forceinline__ void scale32(uint32_t* x, float f) {
  const f2 s = f2_splat(f);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a, b;
    cconv::f2_unpack(f2_mul(s, pair(x, i)), a, b);
    x[2 * i] = __float_as_uint(a);
    x[2 * i + 1] = __float_as_uint(b);
  }
}

// The upper halves of a pair's two words, which are its values cut off to bf16; `rest`: what they leave.
__device__ __forceinline__ uint32_t cut_off(f2 x, f2& rest) {
  float a, b;
  cconv::f2_unpack(x, a, b);
  const uint32_t u = __float_as_uint(a), v = __float_as_uint(b);
  rest = f2_fma(f2_pack(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u)), f2_splat(-1.f), x);
  return __byte_perm(u, v, 0x7632);
}

// A pair's second and third bf16 terms: what its rounding to bf16 leaves has 16 bits at most.
__device__ __forceinline__ void split_rest(f2 s, uint32_t& mid, uint32_t& low) {
  f2 rest = f2_fma(bf16x2_to_f2(f2_to_bf16x2(s)), f2_splat(-1.f), s);
  mid = cut_off(rest, rest);
  low = cut_off(rest, rest);
}

// Scales `width` columns of a TMEM tile in place, a row a thread.
__device__ __forceinline__ void scale_tile(uint32_t tmem, int width, float f) {
#pragma unroll 1
  for (int c = 0; c < width; c += 32) {
    uint32_t x[32];
    tmem_ld32(tmem + c, x);
    tmem_wait_ld();
    tmem_use32(x);
    scale32(x, f);
    tmem_st16(tmem + c, x);
    tmem_st16(tmem + c + 16, x + 16);
  }
  tmem_wait_st();
}

// 128 columns of a TMEM tile, scaled, as bf16 or fp32 rows: to the staging buffer (panels of 128
// bytes a row, 128-byte swizzle) or, for the rows of a partial chunk, straight to memory.
// Columns at or past `width` are left out in steps of 8.
template <bool F32>
__device__ __forceinline__ void finish_tile(uint32_t tmem, uint32_t stage, bool whole, bool live,
                                            int row, int width, float scale, void* dst) {
#pragma unroll 1
  for (int c = 0; c < width; c += 32) {
    uint32_t x[32];
    tmem_ld32(tmem + c, x);
    tmem_wait_ld();
    tmem_use32(x);
    scale32(x, scale);
    if (!F32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = f2_to_bf16x2(pair(x, i));
    }
    constexpr int kPieces = F32 ? 8 : 4, kCols = F32 ? 4 : 8;  // 16-byte pieces of the batch
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = F32 ? i : ((c >> 3) & 7) + i;
      const int panel = F32 ? c >> 5 : c >> 6;
      if (whole)
        sts128(stage + panel * kPanelBytes + swizzled(row, piece), x[4 * i], x[4 * i + 1], x[4 * i + 2],
               x[4 * i + 3]);
      else if (live && c + kCols * i < width)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(dst) + (c + kCols * i) * (F32 ? 4 : 2)) =
            make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
  }
}

// The sums over a key head's members (value heads, column tiles).  Each member's CTA of a cluster
// puts its rows of dq or dk into its ring in fp32, 16 bytes a row side by side, and a chunk later
// adds up its share of the columns from all rings, in the members' order.  Warp by warp, counts in
// every member's shared memory say how many chunks each member has put into its ring.  Two chunks
// are enough for a ring: whoever has counted chunk c has read chunk c - 1.  The rings stay in L2;
// written whole to memory and added up by a kernel of its own, the parts took a third of the time
// (16384 rows, 16 value heads on 8 key heads).
__device__ __forceinline__ void ring_tile(uint32_t tmem, int width, float scale, float4* to) {
#pragma unroll 1
  for (int c = 0; c < width; c += 32) {
    uint32_t x[32];
    tmem_ld32(tmem + c, x);
    tmem_wait_ld();
    tmem_use32(x);
    scale32(x, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + 4 * i < width)
        __stcg(to + (c / 4 + i) * kChunk,
               make_float4(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]),
                           __uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3])));
  }
}
__device__ __forceinline__ void st_pieces(uint16_t* at, const f2* a, const f2* b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(at), "r"(f2_to_bf16x2(a[0])),
               "r"(f2_to_bf16x2(a[1])), "r"(f2_to_bf16x2(a[2])), "r"(f2_to_bf16x2(a[3])),
               "r"(f2_to_bf16x2(b[0])), "r"(f2_to_bf16x2(b[1])), "r"(f2_to_bf16x2(b[2])),
               "r"(f2_to_bf16x2(b[3]))
               : "memory");
}
__device__ __forceinline__ void sum_ring(const float4* from, int group, int pitch, int first, int last,
                                         uint16_t* dst) {
  constexpr int kAt = 2;  // pieces of 8 columns at a time (1 or 4: 4 % slower backward)
#pragma unroll 1
  for (int i = first; i < last; i += kAt) {
    f2 sum[kAt][4];
#pragma unroll
    for (int a = 0; a < kAt * 4; ++a) sum[a / 4][a % 4] = 0;
#pragma unroll 2
    for (int j = 0; j < group; ++j) {
#pragma unroll
      for (int a = 0; a < kAt; ++a) {
        const float4* src = from + j * pitch + 2 * min(i + a, last - 1) * kChunk;
        const float4 x = __ldcg(src), y = __ldcg(src + kChunk);
        sum[a][0] = f2_add(sum[a][0], f2_pack(x.x, x.y));
        sum[a][1] = f2_add(sum[a][1], f2_pack(x.z, x.w));
        sum[a][2] = f2_add(sum[a][2], f2_pack(y.x, y.y));
        sum[a][3] = f2_add(sum[a][3], f2_pack(y.z, y.w));
      }
    }
    uint16_t* at = dst + i * 8;
    if (i + 1 < last && aligned(at, 32)) {
      st_pieces(at, sum[0], sum[1]);
      continue;
    }
#pragma unroll
    for (int a = 0; a < kAt; ++a)
      if (i + a < last)
        *reinterpret_cast<uint4*>(at + a * 8) =
            make_uint4(f2_to_bf16x2(sum[a][0]), f2_to_bf16x2(sum[a][1]), f2_to_bf16x2(sum[a][2]),
                       f2_to_bf16x2(sum[a][3]));
  }
}

template <bool KV, bool FINE>
__global__ void __launch_bounds__(kBwdThreads, 1)
    cattn_linear_chunk_bwd_kernel(const __grid_constant__ BwdArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  Gate* gates = reinterpret_cast<Gate*>(base + kOffGates);
  const uint32_t smem = smem_addr(base);
  const uint32_t full = smem + kOffBars, empty = full + 8 * kBwdSlots;
  const uint32_t gfull = empty + 8 * kBwdSlots, gempty = gfull + 8 * kBwdGates;
  const uint32_t kpfull = gempty + 8 * kBwdGates, kpempty = kpfull + 16;
  const uint32_t fixed = kpempty + 16, scfull = fixed + 8, pfull = scfull + 8, kvfull = pfull + 8;
  const uint32_t kvfree = kvfull + 8, sfull = kvfree + 8, sempty = sfull + 8, infull = sempty + 8;
  const uint32_t scaled = infull + 8, ofull = scaled + 8, ofree = ofull + 8;
  const uint32_t osync = ofree + 8, alldone = osync + 8;  // one for each issuing thread
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(base + kOffBars + 39 * 8);
  const uint32_t stored = smem + kOffBars + 38 * 8;  // chunks whose outputs have left the buffer
  constexpr int kDot = KV ? kK : kQ;  // the tile that the rows' dots read

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBwdSlots; ++i) {
      bar_init(full + 8 * i, 1);
      // readers: the outputs' products, and for one tile each the four warps that take the dots,
      // those that make decayed rows, and (the tile whose rows meet them) the state's products
      const int users = i == kDot || i == (KV ? kQ : kK) ? 5 : i == (KV ? kDo : kV) ? 6 : 1;
      bar_init(empty + 8 * i, users);
    }
    for (int i = 0; i < kBwdGates; ++i) {
      bar_init(gfull + 8 * i, 1);
      bar_init(gempty + 8 * i, kBwdReaders);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(kpfull + 8 * i, 4);
      bar_init(kpempty + 8 * i, 1);
      bar_init(alldone + 8 * i, 1);
    }
    bar_init(fixed, 4);
    bar_init(scfull, 1);
    bar_init(pfull, 4);
    bar_init(kvfull, 1);
    bar_init(kvfree, 4);
    bar_init(sfull, 4);
    bar_init(sempty, 1);
    bar_init(infull, 1);
    bar_init(scaled, KV ? 8 : 4);
    bar_init(ofull, 1);
    bar_init(ofree, 4);
    set_count(stored, 0);
    for (int i = 0; i < 4 * kMaxGroup; ++i) set_count(smem + kOffCounts + 4 * i, 0);
    bar_init(osync, 4);
    cconv::fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_at, 512);
  if (warp == 0 && lane == 0) {
    cconv::prefetch_tensormap(&p.mq);
    cconv::prefetch_tensormap(&p.mk);
    cconv::prefetch_tensormap(&p.mv);
    cconv::prefetch_tensormap(&p.mo);
    cconv::prefetch_tensormap(&p.out_k);
    if (KV) cconv::prefetch_tensormap(&p.out_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const int group = p.plan.group, member = blockIdx.x % group;
  if (group > 1) cluster_sync();  // the counts that the others write are set
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ SmallPlan small;
  Plan plan = p.plan;
  if (plan.small) small_plan(plan, small, false, &g_fault_bwd);

  int nch;
  const int64_t units = unit_count(plan, nch);
  const int64_t parts = range_count(plan, gridDim.x, units);
  const int place = blockIdx.x / group;
  Range range{0, 0};
  if (place < parts) range = range_of(units, parts, place);
  const int count = static_cast<int>(range.u1 - range.u0);
  const int64_t start = KV ? range.u1 - 1 : range.u0;
  const int pk = p.K > kPanelCols ? 2 : 1;
  const uint32_t av = smem + kV * kTileBytes, ao = smem + kDo * kTileBytes;
  const uint32_t ak = smem + kK * kTileBytes, aq = smem + kQ * kTileBytes;

  bool ok = true;  // no wait of this thread's has given up
  if (count > 0) {
  if (warp < 4) {
  // Registers: 96 a thread at the launch, 40 + 120 + 64 + 168 + 88 after.
  set_registers<40, false>();
  if (warp == 0) {
    // ---- tiles ----
    if (elect_one()) {
      Walker w;
      w.seek(&plan, nch, start, member);
      int use = 0, part = 0;
      for (int i = 0; i < count && ok; ++i) {
        if (w.rows() > 0) {
          const int hv = w.ht / plan.tiles, vt = w.ht % plan.tiles;
          const int hk = hv / p.ratio, row = w.row0();
          const int pv = p.V - vt * 128 > kPanelCols ? 2 : 1;
#pragma unroll 1
          for (int j = 0; j < kBwdSlots; ++j) {
            if (use > 0 && !(ok = CATTN_WAIT(empty + 8 * j, use - 1))) break;
            part = j + 1;
            const bool isv = j == kV || j == kDo;
            const CUtensorMap* map = j == kV ? &p.mv : j == kDo ? &p.mo : j == kK ? &p.mk : &p.mq;
            const int panels = isv ? pv : pk;
            bar_expect(full + 8 * j, panels * kPanelBytes);
#pragma unroll 1
            for (int c = 0; c < panels; ++c)
              load_box(smem + j * kTileBytes + c * kPanelBytes, map, full + 8 * j,
                       (isv ? vt * 128 : 0) + c * kPanelCols, isv ? hv : hk, row);
          }
          if (!ok) break;
          ++use;
          part = 0;
        }
        if (i + 1 < count) w.step<KV>();
      }
      for (int j = 0; j < kBwdSlots; ++j) drain(full + 8 * j, use + (j < part ? 1 : 0));
    }
  } else if (warp == 1) {
    // ---- scores, products with the state, and products of P ----
    if (elect_one()) {
      int use = 0, pubs = 0, ins = 0, fixes = 0, kvs = 0;
      const int kk = (p.K + 15) / 16, nk = kk * 16;
      // The rows' dots take the state's product 32 columns at a time: all of these are written (past K
      // with the zeros of the state's rows there), as what an earlier kernel left in tensor memory may
      // be NaN, which the zeros of q or k would not take out.
      const uint32_t ds = mma_desc(128, false, false), dst = mma_desc((p.K + 31) / 32 * 32, false, false);
      const uint32_t dk = mma_desc(nk, false, true);
      const uint64_t tv = tile_desc(av, 0), to = tile_desc(ao, 0), tk = tile_desc(ak, 0);
      const uint64_t tq = tile_desc(aq, 0), tS = tile_desc(smem + kOffS, 0);
      const uint64_t rows_k = tile_desc(KV ? aq : ak, kPanelBytes), rows_o = tile_desc(ao, kPanelBytes);
      const uint64_t tvo = KV ? tv : to;
      const uint64_t rows_S = tile_desc(smem + kOffS, kPanelBytes);
      for (int unit = 0; unit < count && ok; ++unit) {
        const int gs = unit % kBwdGates;
        if (!(ok = CATTN_WAIT(gfull + 8 * gs, unit / kBwdGates))) break;
        const Gate& gt = gates[gs];
        const int n = gt.n, flags = gt.flags;
        if (n > 0) {
          const int kv = (min(128, p.V - gt.ht % plan.tiles * 128) + 15) / 16, nv = kv * 16;
          const int steps = (n + 15) / 16;
          const uint32_t dv = mma_desc(nv, false, true);
#pragma unroll 1
          for (int j = 0; j < kBwdSlots && ok; ++j) ok = CATTN_WAIT(full + 8 * j, use);
          if (!ok) break;
          if (n < kChunk && !(ok = CATTN_WAIT(fixed, fixes++))) break;
          // the score tiles overwrite the last chunk's P (and, for KV, its state product)
          if (use > 0 && !(ok = CATTN_WAIT(ofull, use - 1))) break;
          if (KV && kvs > 0 && !(ok = CATTN_WAIT(kvfree, kvs - 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < kv; ++j)
            mma_ss(tmem, (KV ? tv : to) + col_step(j), (KV ? to : tv) + col_step(j), ds, j > 0);
#pragma unroll 1
          for (int j = 0; j < kk; ++j)
            mma_ss(tmem + 128, (KV ? tk : tq) + col_step(j), (KV ? tq : tk) + col_step(j), ds, j > 0);
          mma_commit(scfull);
          if (!KV) mma_commit(empty + 8 * kQ);
          if (use > 0 && !(ok = CATTN_WAIT(ofree, use - 1))) break;
          const bool has = flags & kHasState;
          if (has) {
            if (!(ok = CATTN_WAIT(sfull, pubs))) break;
            ++pubs;
            tc_fence_after();
            // dO S^T or V D^T: the state's rows are the output's columns, its columns are summed;
            // its small terms first
#pragma unroll 1
            for (int j = 0; j < kv; ++j) mma_ss(tmem + 256, tvo + col_step(j), tS + col_step(j), dst, j > 0);
            mma_commit(sempty);
#pragma unroll 1
            for (int j = 0; j < kv; ++j)
              mma_ss(tmem + 256, tvo + col_step(j), tS + kTileBytes / 16 + col_step(j), dst, true);
            if (!(ok = CATTN_WAIT(sfull, pubs))) break;
            ++pubs;
            tc_fence_after();
#pragma unroll 1
            for (int j = 0; j < kv; ++j) mma_ss(tmem + 256, tvo + col_step(j), tS + col_step(j), dst, true);
            if (KV) {
#pragma unroll 1
              for (int j = 0; j < kk; ++j)
                mma_ss(tmem + 384, tk + col_step(j), rows_S + j * kRowStep, dv, j > 0);
            }
            mma_commit(infull);
            mma_commit(sempty);
            ++ins;
          }
          mma_commit(KV ? empty + 8 * kV : empty + 8 * kDo);
          if (KV) mma_commit(empty + 8 * kK);
          if (!KV) mma_commit(empty + 8 * kV);
          if (!(ok = CATTN_WAIT(pfull, use))) break;
          if (has && !(ok = CATTN_WAIT(scaled, ins - 1))) break;
          tc_fence_after();
          mma_p<FINE>(tmem + 256, tmem, rows_k, dk, steps, has);
          if (KV) mma_p<FINE>(tmem + 384, tmem + 128, rows_o, dv, steps, has);
          mma_commit(ofull);
          mma_commit(empty + 8 * (KV ? kQ : kK));
          if (KV) mma_commit(empty + 8 * kDo);
          if (KV && (flags & kNeedKv)) ++kvs;
          ++use;
        }
        bar_arrive(gempty + 8 * gs);
      }
      mma_commit(alldone);
      drain(alldone, 1);
    }
  } else if (warp == 3) {
    // ---- (kw . K)^T V or (er . Q)^T dO ----
    if (elect_one()) {
      int use = 0, subs = 0, fixes = 0, kvs = 0;
      constexpr int kVals = KV ? kDo : kV;
      const uint64_t rows_v = tile_desc(KV ? ao : av, kPanelBytes);
      for (int unit = 0; unit < count && ok; ++unit) {
        const int gs = unit % kBwdGates;
        if (!(ok = CATTN_WAIT(gfull + 8 * gs, unit / kBwdGates))) break;
        const Gate& gt = gates[gs];
        const int n = gt.n;
        if (n > 0) {
          const int nv = (min(128, p.V - gt.ht % plan.tiles * 128) + 15) / 16 * 16;
          const int steps = (n + 15) / 16;
          if (!(ok = CATTN_WAIT(full + 8 * kVals, use))) break;
          if (n < kChunk && !(ok = CATTN_WAIT(fixed, fixes++))) break;
          // its columns: for KV those of the score tiles, else its own
          if (KV && !(ok = CATTN_WAIT(pfull, use))) break;
          if (gt.flags & kNeedKv) {
            if (!KV && kvs > 0 && !(ok = CATTN_WAIT(kvfree, kvs - 1))) break;
            const uint32_t d0 = mma_desc(KV ? min(nv, 64) : nv, true, true);
            const uint32_t d1 = mma_desc(nv > 64 ? nv - 64 : 16, true, true);
#pragma unroll 1
            for (int b = 0; b < steps; ++b, ++subs) {
              if (!(ok = CATTN_WAIT(kpfull + 8 * (subs & 1), subs >> 1))) break;
              tc_fence_after();
              const uint64_t a = tile_desc(smem + kOffKp + (subs & 1) * kBlockBytes, kBlockPanel);
#pragma unroll
              for (int s = 0; s < kSplit; ++s) {
                mma_ss(tmem + (KV ? 64 : 384), a + s * (kBlockTile / 16), rows_v + b * kRowStep, d0,
                       b + s > 0);
                if (KV && nv > 64)
                  mma_ss(tmem + 192, a + s * (kBlockTile / 16),
                         rows_v + kPanelBytes / 16 + b * kRowStep, d1, b + s > 0);
              }
              mma_commit(kpempty + 8 * (subs & 1));
            }
            if (!ok) break;
            mma_commit(kvfull);
            ++kvs;
            mma_commit(empty + 8 * kVals);
          } else {
            bar_arrive(empty + 8 * kVals);
          }
          ++use;
        }
        bar_arrive(gempty + 8 * gs);
      }
      mma_commit(alldone + 8);
      drain(alldone + 8, 1);
    }
  } else {
    // ---- gates ----
    Walker w;
    w.seek(&plan, nch, start, member);
    for (int unit = 0; unit < count; ++unit) {
      const int gs = unit % kBwdGates, n = w.rows(), row0 = w.row0();
      const int hv = w.ht / plan.tiles;
      float g[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        g[j] = 4 * lane + j < n ? kLog2e * p.g.at(row0 + 4 * lane + j, hv) : 0.f;
      if (unit >= kBwdGates && !(ok = CATTN_WARP_WAIT(gempty + 8 * gs, unit / kBwdGates - 1))) break;
      Gate& gt = gates[gs];
      make_gate(gt, g, lane);
      if (lane == 0) {
        gt.row0 = row0;
        gt.n = n;
        gt.ht = w.ht;
        gt.seq = w.seq;
        int f = 0;
        const bool first = KV ? w.last() : w.first(), last = KV ? w.first() : w.last();
        if (unit == 0 || first) f |= kSegment;
        if ((f & kSegment) && !first) f |= kMiddle;
        if (!first || (!KV && p.initial)) f |= kHasState;
        if (KV && last && p.dinit) f |= kFinish;
        if (KV ? !last || (f & kFinish) : !last && unit + 1 < count) f |= kNeedKv;
        if (KV && !last && unit + 1 == count) f |= kAnchor;
        gt.flags = f;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gfull + 8 * gs);
      if (unit + 1 < count) w.step<KV>();
    }
  }
  } else if (warp < 8) {
    // ---- score tiles to P ----
    set_registers<120, true>();
    const int wq = warp - 4, row = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    int use = 0, pubs = 0;
    for (int unit = 0; unit < count; ++unit) {
      const int gs = unit % kBwdGates;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * gs, unit / kBwdGates))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n;
      if (n > 0) {
        const float own = KV ? gt.ws[row] : gt.lp[row];
        if (!(ok = CATTN_WARP_WAIT(scfull, use))) break;
        tc_fence_after();
        f2 sum = 0;  // pairs of different tokens
        // (P's columns lie in score columns that are read or not needed)
#pragma unroll 1
        for (int b = 0; b < (FINE ? kFineTokens / 32 : 4); ++b) {
          uint32_t x[32], z[32];
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
#pragma unroll 1
            for (int i = lo; i < hi; ++i) e += gt.block[i];
            const f2 ut = f2_splat(KV ? own * exp2_fast(e) : exp2_fast(e));
            const float* cols = (KV ? gt.pe : gt.ws) + b * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(cols + 4 * i);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const f2 wj = f2_mul(ut, j ? w.y : w.x);
                const f2 pj = f2_mul(pair(x, 2 * i + j), wj), zj = pair(z, 2 * i + j);
                sum = f2_fma(pj, zj, sum);
                put_pair(x, 2 * i + j, pj);
                if (KV) put_pair(z, 2 * i + j, f2_mul(zj, wj));
              }
            }
          } else if (b == wq) {
            // the diagonal block: the decay as a running product away from the row's token
            float w = 1.f, s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int i4 = KV ? i : 7 - i;
              const float4 a4 = *reinterpret_cast<const float4*>(&gt.a[b * 32 + 4 * i4]);
              const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
              for (int jj = 0; jj < 4; ++jj) {
                const int j = KV ? jj : 3 - jj, c = 4 * i4 + j;
                const bool off = KV ? c > lane : c < lane, on = off || c == lane;
                if (KV && off) w *= a[j];
                const float v = on ? __uint_as_float(x[c]) * w : 0.f;
                if (off) s = fmaf(v, __uint_as_float(z[c]), s);
                x[c] = __float_as_uint(v);
                if (KV) z[c] = on ? __float_as_uint(__uint_as_float(z[c]) * w) : 0u;
                if (!KV && on) w *= a[j];
              }
            }
            sum = f2_add(sum, f2_pack(s, 0.f));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = z[i] = 0;
          }
          put_p<FINE>(tmem + lanes, b, x);
          if (KV) put_p<FINE>(tmem + lanes + 128, b, z);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(pfull);
        float s0, s1;
        cconv::f2_unpack(sum, s0, s1);
        if (row < n)
          p.dots[static_cast<int64_t>(gt.ht) * p.rows + gt.row0 + row] = p.scale * (s0 + s1);
        ++use;
        if (KV && (gt.flags & kHasState)) {
          // half of the products with the state are scaled here: these warps wait most of the time
          const int vw = min(128, p.V - gt.ht % plan.tiles * 128);
          if (!(ok = CATTN_WARP_WAIT(infull, pubs))) break;
          ++pubs;
          tc_fence_after();
          scale_tile(tmem + lanes + 384, vw, gt.kw[row]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(scaled);
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * gs);
    }
  } else if (warp < 12) {
    // ---- decayed rows ----
    set_registers<64, false>();
    const int kt = threadIdx.x - 256;
    constexpr int kKeys = KV ? kQ : kK, kVals = KV ? kDo : kV;
    const uint32_t src = KV ? aq : ak;
    int use = 0, subs = 0;
    for (int unit = 0; unit < count && ok; ++unit) {
      const int gs = unit % kBwdGates;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * gs, unit / kBwdGates))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n;
      if (n > 0) {
        if (!(ok = CATTN_WARP_WAIT(full + 8 * kKeys, use))) break;
        if (!(ok = CATTN_WARP_WAIT(full + 8 * kVals, use))) break;
        if (n < kChunk) {
          // the tiles whose rows are summed over
          zero_rows(src, pk, n, kt, 128);
          zero_rows(KV ? ao : av, p.V - gt.ht % plan.tiles * 128 > kPanelCols ? 2 : 1, n, kt, 128);
          cconv::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) bar_arrive(fixed);
        }
        if (lane == 0) bar_arrive(empty + 8 * kVals);
        if (gt.flags & kNeedKv) {
          const int steps = (n + 15) / 16;
          const float* weights = KV ? gt.er : gt.kw;
#pragma unroll 1
          for (int b = 0; b < steps; ++b, ++subs) {
            if (subs >= 2 && !(ok = CATTN_WARP_WAIT(kpempty + 8 * (subs & 1), (subs >> 1) - 1))) break;
            const uint32_t dst = smem + kOffKp + (subs & 1) * kBlockBytes;
#pragma unroll 2
            for (int e = kt; e < kBlock * 8 * pk; e += 128) {
              const int r = e >> (2 + pk), piece = e & (8 * pk - 1), t = b * kBlock + r;
              const uint32_t q = piece >> 3, at = swizzled(r, piece & 7);
              uint4 in = lds128_at(src + q * kPanelBytes + b * kBlock * 128 + at);
              if (t >= n) in = make_uint4(0, 0, 0, 0);
              store_split(in, weights[t], dst + q * kBlockPanel + at, kBlockTile);
            }
            cconv::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(kpfull + 8 * (subs & 1));
          }
          if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) bar_arrive(empty + 8 * kKeys);
        ++use;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * gs);
    }
  } else if (warp < 16) {
    // ---- the state: a row of 128 columns a thread ----
    set_registers<168, true>();
    const int krow = threadIdx.x - 384;
    const uint32_t lanes = static_cast<uint32_t>(krow & ~31) << 16;
    f2 S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0;
    int pubs = 0, kvs = 0, done = 0;
    for (int unit = 0; unit < count && ok; ++unit) {
      const int gs = unit % kBwdGates;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * gs, unit / kBwdGates))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, flags = gt.flags;
      const int hv = gt.ht / plan.tiles, vt = gt.ht % plan.tiles;
      const int vw = min(128, p.V - vt * 128);
      if (flags & kSegment) {
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = 0;
        if (flags & kMiddle) {
          // what the ranges before this one (after it, for KV) hand on
          gather_state(S, p.carry, p.decay, blockIdx.x, parts * group, KV ? group : -group, p.joined,
                       krow);
          if (!KV) put_state(S, p.states + static_cast<int64_t>(blockIdx.x) * kStateFloats, krow);
        } else if (!KV && p.initial && krow < p.K) {
          const int64_t slot = p.slots.of(gt.seq);
          const float* src = p.initial + ((slot * p.Hv + hv) * p.K + krow) * p.V + vt * 128;
          if (slot >= 0) load_state(S, src, vw);
        }
      }
      if (n > 0 && (flags & kHasState)) {
        if (pubs > 0 && !(ok = CATTN_WARP_WAIT(sempty, pubs - 1))) break;
        if (!(ok = __all_sync(0xffffffffu, wait_count(stored, done)))) break;
        ++pubs;
        const uint32_t at = smem + kOffS;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t mid[4], low[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) split_rest(S[4 * i + j], mid[j], low[j]);
          const uint32_t to = at + i / 8 * kPanelBytes + swizzled(krow, i % 8);
          sts128(to, mid[0], mid[1], mid[2], mid[3]);
          sts128(to + kTileBytes, low[0], low[1], low[2], low[3]);
        }
        cconv::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(sfull);
        if (!(ok = CATTN_WARP_WAIT(sempty, pubs - 1))) break;  // the middle terms are read
        ++pubs;
        // (rounded anew: kept from above, the first terms would spill)
#pragma unroll
        for (int i = 0; i < 64; ++i) asm volatile("" : "+l"(S[i]));
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sts128(at + i / 8 * kPanelBytes + swizzled(krow, i % 8), f2_to_bf16x2(S[4 * i]),
                 f2_to_bf16x2(S[4 * i + 1]), f2_to_bf16x2(S[4 * i + 2]), f2_to_bf16x2(S[4 * i + 3]));
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
        for (int c = 0; c < 8; ++c) {
          uint32_t x[16];
          tmem_ld16(tmem + lanes + (KV ? (c / 4) * 128 + 64 + (c % 4) * 16 : 384 + c * 16), x);
          tmem_wait_ld();
          tmem_use16(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) S[c * 8 + i] = f2_fma(d, S[c * 8 + i], pair(x, i));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(kvfree);
      }
      if (n > 0) ++done;
      if (KV && (flags & kAnchor)) {
        // dg of the range's first token: the pairs across its start, from both whole states
        const ulonglong2* at = reinterpret_cast<const ulonglong2*>(
            p.states + static_cast<int64_t>(blockIdx.x) * kStateFloats);
        f2 sum = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (krow < p.K && 4 * i < vw) {
            const ulonglong2 x = at[i * 128 + krow];
            sum = f2_fma(S[2 * i], x.x, f2_fma(S[2 * i + 1], x.y, sum));
          }
        float a, b;
        cconv::f2_unpack(sum, a, b);
        a += b;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (lane == 0) p.anchors[blockIdx.x * 4 + krow / 32] = p.scale * a;
      }
      if (KV && (flags & kFinish) && krow < p.K) {
        float* dst = p.dinit + ((static_cast<int64_t>(gt.seq) * p.Hv + hv) * p.K + krow) * p.V + vt * 128;
        const f2 sc = f2_splat(p.scale);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (8 * i < vw) {
            const f2 x[4] = {f2_mul(sc, S[4 * i]), f2_mul(sc, S[4 * i + 1]), f2_mul(sc, S[4 * i + 2]),
                             f2_mul(sc, S[4 * i + 3])};
            st_pairs(dst + 8 * i, x);
          }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * gs);
    }
  } else {
    // ---- the outputs: a row a thread ----
    set_registers<88, false>();
    const int row = threadIdx.x - 512, wq = row / 32;
    const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
    int use = 0, pubs = 0, syncs = 0, last_n = 0, last_row = 0, last_hk = 0;
    // the sums of dq or dk of the last chunk, number use - 1
    auto add_up = [&]() {
      const uint32_t counts = smem + kOffCounts + 4 * (wq * kMaxGroup + lane);
      if (!(ok = __all_sync(0xffffffffu, lane >= group || wait_remote(counts, use)))) return;
      const int pitch = p.K * (kChunk / 4);
      if (row < last_n)
        sum_ring(p.ring + ((blockIdx.x - member) * 2 + (use - 1 & 1)) * pitch + row, group, 2 * pitch,
                 p.K / 8 * member / group, p.K / 8 * (member + 1) / group,
                 p.dqk + (static_cast<int64_t>(last_row + row) * p.Hk + last_hk) * p.K);
      __syncwarp();
    };
    // the four warps meet (with a limit, as every wait)
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(osync);
      return ok = CATTN_WARP_WAIT(osync, syncs++);
    };
    for (int unit = 0; unit < count && ok; ++unit) {
      const int gs = unit % kBwdGates;
      if (!(ok = CATTN_WARP_WAIT(gfull + 8 * gs, unit / kBwdGates))) break;
      const Gate& gt = gates[gs];
      const int n = gt.n, ht = gt.ht, row0 = gt.row0;
      if (n > 0) {
        const int hv = ht / plan.tiles, vt = ht % plan.tiles, vw = min(128, p.V - vt * 128);
        const float rowf = KV ? gt.kw[row] : gt.er[row];
        f2 dot = 0;
        if (!(ok = CATTN_WARP_WAIT(full + 8 * kDot, use))) break;
        if (group > 1) {
          if (use > 0) add_up();
          if (!ok) break;
          last_n = n, last_row = row0, last_hk = hv / p.ratio;
        }
        if (gt.flags & kHasState) {
          if (!(ok = CATTN_WARP_WAIT(infull, pubs))) break;
          ++pubs;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < p.K; c += 32) {
            uint32_t x[32];
            tmem_ld32(tmem + lanes + 256 + c, x);
            tmem_wait_ld();
            tmem_use32(x);
            dot = dot_tile(KV ? ak : aq, row, c, x, dot);
            scale32(x, rowf);
            tmem_st16(tmem + lanes + 256 + c, x);
            tmem_st16(tmem + lanes + 256 + c + 16, x + 16);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(scaled);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(empty + 8 * kDot);
        const int64_t t = row0 + row;
        float d0, d1;
        cconv::f2_unpack(dot, d0, d1);
        if (row < n)
          p.dots[(static_cast<int64_t>(plan.heads) * plan.tiles + ht) * p.rows + t] =
              p.scale * rowf * (d0 + d1);
        if (!(ok = CATTN_WARP_WAIT(ofull, use))) break;
        // The last chunk's outputs may still be on their way out of the staging buffer: `ofree` does
        // not wait for them, and only a chunk with a state is held back by the state's warps.  (In a
        // cluster they have left before `ofree`.)
        if (group == 1 && !(ok = __all_sync(0xffffffffu, wait_count(stored, use)))) break;
        tc_fence_after();
        const bool whole = n == kChunk, live = row < n;
        const int hk = hv / p.ratio;
        const uint32_t stage = smem + kOffS;
        if (group == 1) {
          if (p.part)
            finish_tile<true>(tmem + lanes + 256, stage, whole, live, row, p.K, p.scale,
                              p.part + (static_cast<int64_t>(ht) * p.rows + t) * p.K);
          else
            finish_tile<false>(tmem + lanes + 256, stage, whole, live, row, p.K, p.scale,
                               p.dqk + (t * p.Hk + hk) * p.K);
          if (whole) {
            cconv::fence_proxy_async_smem();
            if (!meet()) break;
            if (row == 0) {
              const int cols = p.part ? 32 : 64;
#pragma unroll 1
              for (int c = 0, i = 0; c < p.K; c += cols, ++i)
                store_box(&p.out_k, stage + i * kPanelBytes, c, p.part ? ht : hk, row0);
              stores_commit();
              if (KV) stores_wait_read();
            }
            if (KV && !meet()) break;
          }
        }
        if (KV) {
          finish_tile<false>(tmem + lanes + 384, stage, whole, live, row, vw, p.scale,
                             p.dv + (t * p.Hv + hv) * p.V + vt * 128);
          if (whole) {
            cconv::fence_proxy_async_smem();
            if (!meet()) break;
            if (row == 0) {
#pragma unroll 1
              for (int c = 0, i = 0; c < vw; c += 64, ++i)
                store_box(&p.out_v, stage + i * kPanelBytes, vt * 128 + c, hv, row0);
              stores_commit();
            }
          }
        }
        // the state may have its buffer back: in a cluster before the ring is written (2 % of the
        // sweep of 16384 rows against after it)
        auto leave = [&]() {
          if (row != 0) return;
          stores_wait_read();
          set_count(stored, use + 1);
        };
        if (group > 1) {
          leave();
          __syncwarp();
          ring_tile(tmem + lanes + 256, p.K, p.scale,
                    p.ring + (blockIdx.x * 2 + (use & 1)) * (p.K * (kChunk / 4)) + row);
          __syncwarp();
          if (lane < group) set_remote(smem + kOffCounts + 4 * (wq * kMaxGroup + member), lane, use + 1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(ofree);
        if (group == 1) leave();
        ++use;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(gempty + 8 * gs);
    }
    if (ok && group > 1 && use > 0) add_up();
    if (row == 0) stores_wait();  // all of it is written
  }
  }
  if (!ok) atomicOr(&g_fault_bwd, kFaultWait);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  if (group > 1) cluster_sync();  // no member's counts arrive after this CTA has gone
}

static cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&attr)[2], int grid, int group,
                                         cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = group, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid), lc.blockDim = dim3(kBwdThreads);
  lc.dynamicSmemBytes = kBwdBytes, lc.stream = stream;
  lc.attrs = attr, lc.numAttrs = 2;
  return lc;
}

template <bool KV>
static int launch_sweep(const BwdArgs& a, int grid, cudaStream_t stream) {
  auto kern = a.rows <= kFineTokens ? cattn_linear_chunk_bwd_kernel<KV, true> : cattn_linear_chunk_bwd_kernel<KV, false>;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kBwdBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  if (a.plan.group == 1 || cconv::recording_launches())
    return launch_pdl(kern, dim3(grid), dim3(kBwdThreads), kBwdBytes, stream, a) == cudaSuccess
               ? CCONV_OK
               : CCONV_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = cluster_config(attr, grid, a.plan.group, stream);
  return report_cuda("kernel launch", cudaLaunchKernelEx(&lc, kern, a)) == cudaSuccess ? CCONV_OK
                                                                                      : CCONV_ERR_CUDA;
}

int cluster_ctas(int group, int* ctas) {
  // asked once for each size and device (0: not yet)
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxGroup + 1];
  int device = 0;
  if (report_cuda("cudaGetDevice", cudaGetDevice(&device)) != cudaSuccess) return CCONV_ERR_CUDA;
  std::atomic<int>* at = device < kDevices ? &known[device][group] : nullptr;
  if (at && (*ctas = at->load(std::memory_order_relaxed)) > 0) return CCONV_OK;
  auto kern = cattn_linear_chunk_bwd_kernel<true, false>;
  if (cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kern), kBwdBytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t lc = cluster_config(attr, group, group, nullptr);
  int clusters = 0;
  if (report_cuda("cluster occupancy", cudaOccupancyMaxActiveClusters(&clusters, kern, &lc)) != cudaSuccess)
    return CCONV_ERR_CUDA;
  *ctas = clusters * group;
  if (at) at->store(*ctas, std::memory_order_relaxed);
  return CCONV_OK;
}

size_t sum_bytes(int grid, int64_t K) { return static_cast<size_t>(grid) * 2 * kChunk * K * sizeof(float); }

// Map of dq or dk, or of their parts.
static int out_map(CUtensorMap* map, uint16_t* d, float* part, const ChunkBwdCall& c) {
  const int tiles = (c.s.V + 127) / 128;
  if (part) return encode_part_map(map, part, c.s.total, int64_t(c.s.Hv) * tiles, c.s.K);
  return encode_tile_map(map, Rows{d, int64_t(c.s.Hk) * c.s.K, c.s.K}, c.s.total, c.s.Hk, c.s.K);
}

int launch_chunk_bwd(const ChunkBwdCall& c, cudaStream_t stream) {
  BwdArgs a{};
  int rc = encode_tile_map(&a.mq, c.q, c.s.total, c.s.Hk, c.s.K);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mk, c.k, c.s.total, c.s.Hk, c.s.K);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mv, c.v, c.s.total, c.s.Hv, c.s.V);
  if (rc == CCONV_OK) rc = encode_tile_map(&a.mo, c.d_o, c.s.total, c.s.Hv, c.s.V);
  if (rc == CCONV_OK)
    rc = encode_tile_map(&a.out_v, Rows{c.dv, int64_t(c.s.Hv) * c.s.V, c.s.V}, c.s.total, c.s.Hv, c.s.V);
  if (rc == CCONV_OK) rc = out_map(&a.out_k, c.dq, c.part_q, c);
  if (rc != CCONV_OK) return rc;
  const int tiles = (c.s.V + 127) / 128;
  a.plan = Plan{c.cu, c.cstart, c.s.nseq, tiles, c.s.Hv, c.group, c.cstart == nullptr, c.s.total, nullptr, 0,
                nullptr};
  a.g = c.g;
  a.slots = c.slots;
  a.initial = c.initial;
  a.dinit = c.dinit;
  a.dqk = c.dq, a.dv = c.dv;
  a.scale = c.scale;
  a.rows = c.s.total, a.ratio = c.s.Hv / c.s.Hk;
  a.joined = c.joined;
  a.Hk = c.s.Hk, a.Hv = c.s.Hv, a.K = c.s.K, a.V = c.s.V;
  a.carry = c.carry_s;
  a.decay = c.carry_s + static_cast<int64_t>(c.grid) * 2 * kStateFloats;
  a.part = c.part_q, a.dots = c.dots_q;
  a.ring = reinterpret_cast<float4*>(c.ring);
  // (the hand-on kernels use neither of these for the backward)
  a.states = c.carry_s + static_cast<int64_t>(c.grid) * kStateFloats;
  a.anchors = c.carry_d + static_cast<int64_t>(c.grid) * kStateFloats;
  rc = launch_sweep<false>(a, c.grid, stream);
  if (rc == CCONV_OK) rc = out_map(&a.out_k, c.dk, c.part_k, c);
  if (rc != CCONV_OK) return rc;
  a.dqk = c.dk;
  a.carry = c.carry_d;
  a.decay = c.carry_d + static_cast<int64_t>(c.grid) * 2 * kStateFloats;
  a.part = c.part_k, a.dots = c.dots_k;
  return launch_sweep<true>(a, c.grid, stream);
}

}  // namespace cattn
