// attn_chunk.cuh -- how the chunked linear attention divides its work, and the pieces its
// kernels share.
//
// A sequence is cut into chunks of 128 tokens.  The units of work are (value head, column tile
// of V, chunk), ordered so that the chunks of one head follow one another; each CTA takes one
// contiguous range of units, equal to within one unit whatever the lengths of the sequences
// are.  A range that ends inside a sequence hands its state on through the workspace.
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
constexpr int kStateFloats = 128 * 128;        // a state in the workspace

// Chunk offsets of the sequences: cstart[nseq + 1], an empty sequence has one (empty) chunk.
struct Plan {
  const int32_t* cu;
  const int32_t* cstart;
  int nseq;
  int tiles;  // column tiles of V
  int heads;  // value heads
};

struct Range {
  int64_t u0, u1;  // units of this CTA, [u0, u1)
};

// The part of a range that continues in the next range (the previous one for a sweep from the
// last token): [u0, u1), empty if the range's end is a sequence's end; `closed` if the sequence
// starts (ends) in this range.
struct Tail {
  int64_t u0, u1;
  bool closed;
};

__device__ __forceinline__ int64_t unit_count(const Plan& p, int& nch) {
  nch = p.cstart[p.nseq];
  return static_cast<int64_t>(p.heads) * p.tiles * nch;
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
  __device__ __forceinline__ void seek(const Plan* plan, int chunks, int64_t u) {
    p = plan;
    nch = chunks;
    ht = static_cast<int>(u / nch);
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
      ++ht;
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
      --ht;
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
};

__device__ __forceinline__ float shfl_scan_up(float x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ float shfl_scan_down(float x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_down_sync(0xffffffffu, x, o);
    if (lane + o < 32) x += y;
  }
  return x;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void make_gate(Gate& s, const float (&g)[4], int lane) {
  float pre[4], post[4], tot[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    pre[b] = shfl_scan_up(g[b], lane);
    const float after = __shfl_down_sync(0xffffffffu, g[b], 1);
    post[b] = shfl_scan_down(lane == 31 ? 0.f : after, lane);
    tot[b] = __shfl_sync(0xffffffffu, pre[b], 31);
  }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float before = 0.f, behind = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < b) before += tot[i];
      if (i > b) behind += tot[i];
    }
    const int t = 32 * b + lane;
    s.a[t] = exp2_fast(g[b]);
    s.ws[t] = exp2_fast(post[b]);
    s.lp[t] = pre[b];
    s.pe[t] = exp2_fast(pre[b]);
    s.er[t] = exp2_fast(pre[b] + before);
    s.kw[t] = exp2_fast(post[b] + behind);
  }
  if (lane < 4) s.block[lane] = lane == 0 ? tot[0] : lane == 1 ? tot[1] : lane == 2 ? tot[2] : tot[3];
  if (lane == 0) s.total = exp2_fast(tot[0] + tot[1] + tot[2] + tot[3]);
}

// Waits for a phase of `bar`, at most kWaitLimitNs; gives up at once where another role of the
// CTA has.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                           unsigned* fault) {
  if (cconv::mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = cconv::global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    if (cconv::mbar_try_wait(bar, parity)) return true;
    if ((n & 63u) == 0 && (*gave_up || cconv::global_timer_ns() - t0 > cconv::kWaitLimitNs)) {
      *gave_up = 1;
      atomicOr(fault, kFaultWait);
      return false;
    }
  }
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

// x rounded to bf16 three times: x = hi + mid + lo to 24 bits.  Eight values at a time.
__device__ __forceinline__ void split3(const float* x, uint32_t* hi, uint32_t* mid, uint32_t* lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
    const uint32_t h = pack_bf16(a, b);
    a -= __uint_as_float(h << 16);
    b -= __uint_as_float(h & 0xffff0000u);
    const uint32_t m = pack_bf16(a, b);
    a -= __uint_as_float(m << 16);
    b -= __uint_as_float(m & 0xffff0000u);
    hi[i] = h;
    mid[i] = m;
    lo[i] = pack_bf16(a, b);
  }
}

}  // namespace cattn
