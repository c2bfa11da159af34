// attn_chunk.cuh -- how the chunked linear attention divides its work, and the pieces its
// kernels share.
//
// A sequence is cut into chunks of 128 tokens.  The units of work are (value head, column tile
// of V, chunk), ordered so that the chunks of one head follow one another; each CTA takes one
// contiguous range of units, equal to within one unit whatever the lengths of the sequences
// are.  A range that ends inside a sequence hands its state on through the workspace.
//
// Where the sums over the value heads (and column tiles) of one key head are made by the CTAs of a
// cluster, such a group of `group` neighbours shares one range of (key head, chunk), and each takes
// one of its members: range i of member m is CTA i * group + m.
#pragma once

#include "attn_tc.cuh"

namespace cattn {

constexpr int kChunk = 128;
constexpr int kTileBytes = kChunk * 128 * 2;   // a [128 tokens, 128 channels] tile
constexpr int kPanelBytes = kChunk * 128;      // its 64-column panels
constexpr int kSub = 32;                       // tokens of one decayed block of keys
constexpr int kSplit = 3;                      // bf16 terms of a decayed key: 24 bits
constexpr int kSubPanel = kSub * 128;          // bytes of a block's 64-column panel
constexpr int kSubTile = 2 * kSubPanel;
constexpr int kSubBytes = kSplit * kSubTile;
constexpr int kGateStages = 3;
constexpr int kRowStep = 16 * 128 / 16;        // descriptor units (16 bytes) of 16 tile rows

// Descriptor offset of 16 columns' step j of a tile (columns as the contraction).
__device__ __forceinline__ uint64_t col_step(int j) {
  return static_cast<uint64_t>((j >> 2) * (kPanelBytes / 16) + (j & 3) * 2);
}

constexpr int kStateFloats = 128 * 128;        // a state in the workspace
// In place of the decay of what a range hands on: its sequence starts (ends) there; nothing is
// handed on.
constexpr float kChainStart = -1.f, kNoTail = -2.f;

// Chunk offsets of the sequences: cstart[nseq + 1], an empty sequence has one (empty) chunk.
// Up to kSmallPlan sequences, every CTA makes them itself (small_plan), with the checks of the
// row offsets and state indices: that costs less than a launch before the kernels.
struct Plan {
  const int32_t* cu;
  const int32_t* cstart;
  int nseq;
  int tiles;  // column tiles of V
  int heads;  // value heads
  int group;  // CTAs that share a range: 1, or the members of a key head
  int small, total;
  const int32_t* idx;  // state indices, their slots, and where the verdict goes
  int64_t S;
  int32_t* status;
};
constexpr int kSmallPlan = 32;
struct SmallPlan {
  int32_t cu[kSmallPlan + 1], cstart[kSmallPlan + 1];
  int32_t usable;  // the state indices are
};

// All threads of the CTA; ends with a barrier.  `report`: this CTA writes the verdicts.
__device__ __forceinline__ void small_plan(Plan& p, SmallPlan& s, bool report, unsigned* fault) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int a = lane < p.nseq ? p.cu[lane] : 0, b = lane < p.nseq ? p.cu[lane + 1] : 0;
    bool bad = lane < p.nseq && (b < a || (lane == 0 && a != 0) || (lane == p.nseq - 1 && b != p.total));
    bad = __any_sync(0xffffffffu, bad);
    int x = lane < p.nseq && !bad ? max(1, (b - a + kChunk - 1) / kChunk) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane < p.nseq) {
      s.cu[lane] = a;
      s.cu[lane + 1] = b;  // (lane + 1 writes the same value)
      s.cstart[lane + 1] = x;
    }
    unsigned off = 0;
    if (p.idx) off = check_indices(lane < p.nseq ? p.idx[lane] : -1, p.nseq, p.S, false, lane);
    if (lane == 0) {
      s.cstart[0] = 0;
      s.usable = off == 0;
      if (report) {
        if (bad) atomicOr(fault, kFaultSeqlens);
        if (p.idx) {
          p.status[0] = off ? CCONV_ERR_INDEX : CCONV_OK;
          p.status[1] = static_cast<int>(off);
        }
      }
    }
  }
  __syncthreads();
  p.cu = s.cu;
  p.cstart = s.cstart;
}

struct Range {
  int64_t u0, u1;  // units of this CTA, [u0, u1)
};
// How many ranges there are.
__device__ __forceinline__ int64_t range_count(const Plan& p, int64_t grid, int64_t units) {
  const int64_t ranges = grid / p.group;
  return ranges < units ? ranges : units;
}

// The part of a range that continues in the next range (the previous one for a sweep from the
// last token): [u0, u1), empty if the range's end is a sequence's end; `closed` if the sequence
// starts (ends) in this range.
struct Tail {
  int64_t u0, u1;
  bool closed;
};

__device__ __forceinline__ int64_t unit_count(const Plan& p, int& nch) {
  nch = p.cstart[p.nseq];
  return static_cast<int64_t>(p.heads) * p.tiles / p.group * nch;
}
__device__ __forceinline__ Range range_of(int64_t units, int64_t parts, int64_t i) {
  return Range{units * i / parts, units * (i + 1) / parts};
}

// Walks a CTA's units.
struct Walker {
  const Plan* p;
  int nch, ht;           // chunks of all sequences; head * tiles + tile
  int c, seq;            // chunk and its sequence
  int cs, ce, base, len; // the sequence's chunks and rows

  __device__ __forceinline__ void load() {
    cs = p->cstart[seq];
    ce = p->cstart[seq + 1];
    base = p->cu[seq];
    len = p->cu[seq + 1] - base;
  }
  __device__ __forceinline__ void seek(const Plan* plan, int chunks, int64_t u, int member = 0) {
    p = plan;
    nch = chunks;
    ht = static_cast<int>(u / nch) * p->group + member;
    c = static_cast<int>(u % nch);
    int lo = 0, hi = p->nseq - 1;  // the last sequence whose first chunk is <= c
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p->cstart[mid] <= c)
        lo = mid;
      else
        hi = mid - 1;
    }
    seq = lo;
    load();
  }
  __device__ __forceinline__ void next() {
    ++c;
    if (c == nch) {
      c = 0;
      seq = 0;
      ht += p->group;
      load();
    } else if (c == ce) {
      ++seq;
      load();
    }
  }
  __device__ __forceinline__ void prev() {
    --c;
    if (c < 0) {
      c = nch - 1;
      seq = p->nseq - 1;
      ht -= p->group;
      load();
    } else if (c < cs) {
      --seq;
      load();
    }
  }
  template <bool REV>
  __device__ __forceinline__ void step() {
    if (REV)
      prev();
    else
      next();
  }
  __device__ __forceinline__ bool first() const { return c == cs; }
  __device__ __forceinline__ bool last() const { return c == ce - 1; }
  __device__ __forceinline__ int row0() const { return base + (c - cs) * kChunk; }
  __device__ __forceinline__ int rows() const { return min(kChunk, len - (c - cs) * kChunk); }
};

template <bool REV>
__device__ __forceinline__ Tail tail_of(const Plan& p, int nch, int64_t units, const Range& r) {
  Tail t{r.u1, r.u1, false};
  if (r.u0 >= r.u1) return t;
  Walker w;
  if (!REV) {
    if (r.u1 == units) return t;
    w.seek(&p, nch, r.u1);
    if (w.first()) return t;
    const int64_t began = r.u1 - (w.c - w.cs);
    t.closed = began >= r.u0;
    t.u0 = t.closed ? began : r.u0;
  } else {
    if (r.u0 == 0) return t;
    w.seek(&p, nch, r.u0);
    if (w.first()) return t;
    const int64_t ends = r.u0 + (w.ce - w.c);
    t.closed = ends <= r.u1;
    t.u0 = r.u0;
    t.u1 = t.closed ? ends : r.u1;
  }
  return t;
}

// One chunk's gates, made by one warp for the others.  All exponents are sums of gates of one
// sign, never differences of running sums, so that the factors are accurate to a few 2^-22
// whatever the decays are.
struct alignas(16) Gate {
  float a[kChunk];     // exp(g_t)
  float ws[kChunk];    // decay from token s to the end of its block of 32
  float lp[kChunk];    // log2 of the decay from before the block to token t
  float er[kChunk];    // decay from before the chunk to token t
  float kw[kChunk];    // decay from token s to the end of the chunk
  float pe[kChunk];    // decay from before the block to token t
  float block[4];      // log2 decay of each block
  float total;         // decay of the chunk
  int row0, n, ht, seq, flags;
};
enum GateFlags : int {
  kSegment = 1,   // a state is (re)loaded before this chunk
  kMiddle = 2,    // and comes from the ranges before this one
  kHasState = 4,  // the state before this chunk is not known to be zero
  kNeedKv = 8,    // the state after it is needed
  kFinish = 16,   // and it is the sequence's last: a final state
  kSplitSeq = 32, // this sequence began in this range and goes on in the next
  kAnchor = 64,   // the range's first unit, inside a sequence
};

using cconv::f2;
using cconv::f2_add;
using cconv::f2_fma;
using cconv::f2_mul;
using cconv::f2_pack;
using cconv::f2_splat;
using cconv::f2_to_bf16x2;
using cconv::bf16x2_to_f2;

__device__ __forceinline__ f2 pair(const uint32_t* x, int i) {
  return f2_pack(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
}

constexpr float kLog2e = 1.4426950408889634f;

// g: the log2 decays of tokens 4 lane .. 4 lane + 3; a block of 32 tokens is 8 lanes.
__device__ __forceinline__ void make_gate(Gate& s, const float (&g)[4], int lane) {
  const float own = (g[0] + g[1]) + (g[2] + g[3]);
  // sums over the block's lanes before and after this one, and over the chunk's blocks
  float before = 0.f, after = 0.f, up = own, down = own;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, up, o, 8), y = __shfl_down_sync(0xffffffffu, down, o, 8);
    if ((lane & 7) >= o) up += x;
    if ((lane & 7) + o < 8) down += y;
  }
  const float x = __shfl_up_sync(0xffffffffu, up, 1, 8), y = __shfl_down_sync(0xffffffffu, down, 1, 8);
  if ((lane & 7) > 0) before = x;
  if ((lane & 7) < 7) after = y;
  float head = 0.f, rest = 0.f, all = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float t = __shfl_sync(0xffffffffu, down, 8 * b);
    if (b < lane / 8) head += t;
    if (b > lane / 8) rest += t;
    all += t;
    if (lane == 0) s.block[b] = t;
  }
  float pre[4], post[4];
  pre[0] = before + g[0], pre[1] = pre[0] + g[1], pre[2] = pre[1] + g[2], pre[3] = pre[2] + g[3];
  post[3] = after, post[2] = after + g[3], post[1] = post[2] + g[2], post[0] = post[1] + g[1];
  float v[6][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[0][j] = exp2_fast(g[j]);
    v[1][j] = exp2_fast(post[j]);
    v[2][j] = pre[j];
    v[3][j] = exp2_fast(head + pre[j]);
    v[4][j] = exp2_fast(post[j] + rest);
    v[5][j] = exp2_fast(pre[j]);
  }
  float* rows = s.a;  // a, ws, lp, er, kw, pe follow one another
#pragma unroll
  for (int i = 0; i < 6; ++i)
    *reinterpret_cast<float4*>(rows + i * kChunk + 4 * lane) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
  if (lane == 0) s.total = exp2_fast(all);
}

// Tries of one wait: some tenths of a second at least, against waits of microseconds.
constexpr int kWaitTries = 1 << 22;

// The loads of a tile slot must have landed before a CTA's shared memory goes: waits for the last
// of `uses` phases of `full`, with a limit.
__device__ __forceinline__ void drain(uint32_t full, int uses) {
#pragma unroll 1
  for (int n = kWaitTries / 16; uses > 0 && n != 0; --n)
    if (bar_try(full, static_cast<uint32_t>(uses - 1) & 1u)) return;
}

// Waits for a phase of `bar`; false when it gives up (then the role ends, and the roles that wait
// for it give up in their turn).  Kept short: it is inlined at every wait, and the kernels' loops
// have to fit the instruction cache.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int n = kWaitTries; n != 0; --n)
    if (bar_try(bar, parity)) return true;
  return false;
}

// How the roles of a kernel meet: an mbarrier wait tells an odd phase from an even one only, so
// a role (1) waits for every phase of a barrier that it uses, in order, needed or not, and (2)
// holds back the phase after the one it waits for (whoever waits for a tile also gives it back).
// Where a role follows another that it does not hold back, it follows a counter:

__device__ __forceinline__ void set_count(uint32_t at, int value) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(at), "r"(value) : "memory");
}
// Waits until the count reaches `value`; false when it gives up.
__device__ __forceinline__ bool wait_count(uint32_t at, int value) {
#pragma unroll 1
  for (int n = kWaitTries; n != 0; --n) {
    int now;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(now) : "r"(at) : "memory");
    if (now >= value) return true;
  }
  return false;
}

// The same between the CTAs of a cluster: a count in the shared memory of CTA `rank`, and the wait
// for a count that another one sets.  What the writer did before is seen after the wait.
__device__ __forceinline__ void set_remote(uint32_t at, int rank, int value) {
  uint32_t there;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("st.release.cluster.shared::cluster.b32 [%0], %1;" ::"r"(there), "r"(value) : "memory");
}
__device__ __forceinline__ bool wait_remote(uint32_t at, int value) {
#pragma unroll 1
  for (int n = kWaitTries; n != 0; --n) {
    int now;
    asm volatile("ld.acquire.cluster.shared::cta.b32 %0, [%1];" : "=r"(now) : "r"(at) : "memory");
    if (now >= value) return true;
  }
  return false;
}

// Zeroes rows [n, 128) of a tile: rows of the next sequence must not meet a matrix product,
// where 0 * NaN is not 0.  `threads` threads, i of them this one.
__device__ __forceinline__ void zero_rows(uint32_t tile, int panels, int n, int i, int threads) {
  const int pieces = (kChunk - n) * 8;
  for (int e = i; e < panels * pieces; e += threads) {
    const int panel = e / pieces, at = e % pieces;
    sts128(tile + panel * kPanelBytes + (n + at / 8) * 128 + (at % 8) * 16, 0, 0, 0, 0);
  }
}

// S (a row of 64 pairs) to the workspace, 16 bytes a lane side by side.
__device__ __forceinline__ void put_state(const f2* S, float* dst, int row) {
  ulonglong2* to = reinterpret_cast<ulonglong2*>(dst);
#pragma unroll
  for (int i = 0; i < 32; ++i) to[i * 128 + row] = make_ulonglong2(S[2 * i], S[2 * i + 1]);
}

// A row of a state in memory, `width` of its columns.
__device__ __forceinline__ void load_state(f2* S, const float* src, int width) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    Pairs4 x{};
    if (8 * i < width) x = ld_pairs(src + 8 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) S[4 * i + j] = x.v[j];
  }
}

// Adds up what the ranges next to CTA `at`'s hand on (by < 0: those before it, > 0: after it; by
// the CTAs of a range), to the one where the sequence starts (ends); the nearest one's is the
// whole where they are joined.
__device__ __forceinline__ void gather_state(f2* S, const float* carry, const float* decay,
                                             int64_t at, int64_t ctas, int by, bool joined,
                                             int row) {
  float coef = 1.f;
  for (int64_t j = at + by; j >= 0 && j < ctas; j += by) {
    const ulonglong2* src = reinterpret_cast<const ulonglong2*>(carry + j * kStateFloats);
    const float d = decay[j];
    const f2 c = f2_splat(coef);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const ulonglong2 x = src[i * 128 + row];
      S[2 * i] = f2_fma(c, x.x, S[2 * i]);
      S[2 * i + 1] = f2_fma(c, x.y, S[2 * i + 1]);
    }
    if (joined || d < 0.f) break;
    coef *= d;
    if (coef == 0.f) break;
  }
}

// Calls of at most 64 rows keep P in two bf16 terms (FINE kernels).  Over a few tokens the rounding of
// single scores does not average out (up to 1.75 times the error of the bf16 store; with more tokens it
// is 1.4 times that whatever the inputs are).  What that turns on is the length of each sequence, which
// the host does not know: 64 rows is the largest call that is sure to have no longer chunk, and for
// longer ones the dk, dv sweep has no room (D's product takes columns 64 to 127 of each score tile).
// So a short sequence in a call of more than 64 rows has its scores in one term, like the long ones
// beside it.  64 tokens take 7.7 us with two terms and with one; decided chunk by chunk, the larger
// calls paid for it: 112 us against 110 for 16384 rows, 416 against 384 for their gradient.  (The state
// that the forward's Q S reads has one term in every call.)  Columns of TMEM: block b's first terms at
// 32 b and its second ones 16 on, over scores that are read; with one term at 16 b.
constexpr int kFineTokens = 64;

// P times `steps` rows of 16 tokens at `rows`, onto `out` (from zero unless `add`).
template <bool FINE>
__device__ __forceinline__ void mma_p(uint32_t out, uint32_t p, uint64_t rows, uint32_t desc, int steps,
                                      bool add) {
#pragma unroll 1
  for (int j = 0; j < (FINE ? 2 * steps : steps); ++j) {
    const int step = FINE ? j >> 1 : j;
    mma_ts(out, p + (FINE ? (step >> 1) * 32 + (step & 1) * 8 + (j & 1) * 16 : j * 8), rows + step * kRowStep,
           desc, add || j > 0);
  }
}
template <bool FINE>
__device__ __forceinline__ void put_p(uint32_t tmem, int b, const uint32_t (&x)[32]) {
  uint32_t y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = f2_to_bf16x2(pair(x, i));
  tmem_st16(tmem + b * (FINE ? 32 : 16), y);
  if (!FINE) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = f2_to_bf16x2(f2_fma(bf16x2_to_f2(y[i]), f2_splat(-1.f), pair(x, i)));
  tmem_st16(tmem + b * 32 + 16, y);
}
__device__ __forceinline__ void put_pair(uint32_t (&x)[32], int i, f2 v) {
  float a, b;
  cconv::f2_unpack(v, a, b);
  x[2 * i] = __float_as_uint(a), x[2 * i + 1] = __float_as_uint(b);
}

// Eight bf16 values times w, each rounded to bf16 three times: x = hi + mid + lo to 24 bits.
// The three terms of 16 bytes go to `at`, at + step and at + 2 step.
__device__ __forceinline__ void store_split(const uint4& in, float w, uint32_t at, uint32_t step) {
  const uint32_t word[4] = {in.x, in.y, in.z, in.w};
  const f2 w2 = f2_splat(w), minus = f2_splat(-1.f);
  uint32_t t[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2 x = f2_mul(bf16x2_to_f2(word[i]), w2);
    t[0][i] = f2_to_bf16x2(x);
    x = f2_fma(bf16x2_to_f2(t[0][i]), minus, x);
    t[1][i] = f2_to_bf16x2(x);
    x = f2_fma(bf16x2_to_f2(t[1][i]), minus, x);
    t[2][i] = f2_to_bf16x2(x);
  }
#pragma unroll
  for (int s = 0; s < kSplit; ++s) sts128(at + s * step, t[s][0], t[s][1], t[s][2], t[s][3]);
}

}  // namespace cattn
