// attn_delta.cuh -- how the gated delta rule is computed, and what its kernels share.
//
//   S_t = e^{g_t} S_{t-1} + k_t u_t^T,  u_t = beta_t z_t,  z_t = v_t - (e^{g_t} S_{t-1})^T k_t
//   o_t = scale q_t^T S_t
//
// Given u this is linear attention with decay.  In a chunk of 64 tokens that starts from S_0, with
// L_ts the decay from token s to token t, ef_t that from before the chunk to t and eb_t that from t
// to the chunk's end, M = strictly lower (K K^T . L), P = lower (Q K^T . L) and B = diag(beta):
//
//   (1 + M B) z = r = v - ef . (K S_0)
//   J  = -M (1 + B M)^-1  (strictly lower)      z = r + J (B r),  u = B z
//   P~ =  P (1 + B M)^-1                        P u = P~ (B r)
//   o  = scale (ef . (Q S_0) + P~ (B r)),       S_1 = total S_0 + K^T (eb . u)
//
// J holds for beta = 0 as well, and serves the gradient with its transpose (D: the gradient of the
// state at the chunk's end, r' = eb . (K D)):
//
//   du = r' + J^T (B r') + scale P~^T do,  dv = B du,  dbeta = du . z
//   D_0 = total D + scale Q^T (ef . do) - K^T (ef . dv)
//
// J, P~ and the gates depend on q, k, g and beta only: a first kernel makes them for all chunks at
// once (attn_delta_prep.cu) and leaves them in the workspace, a record for each chunk and value head.
// What is left is a chain over the chunks of a sequence, whose columns of V are independent
// (attn_delta_chain.cuh): a CTA takes 32 of them.
//
// Precision: products run on bf16 with fp32 accumulators; an fp32 factor is split into three bf16
// terms (24 bits), and for two such factors the products of terms down to 2^-16 are summed.  (Two terms, 16 bits, in
// a forward that leaves no state saved a tenth of its time, and its o differed from that of the same call
// with a final state.)
#pragma once

#include "attn_chunk.cuh"

namespace cattn {

constexpr int kDelta = 64;                         // tokens of a chunk
constexpr int kTerms = 3;                          // bf16 terms of an fp32 factor
constexpr int kSideBytes = kDelta * 128;           // 64 rows of a 64-column panel
constexpr int kPieceBytes = 128 * 16;              // 8 columns (16 bytes a row) of J's and P~'s rows
constexpr int kTermBytes = 8 * kPieceBytes;        // one term of them
constexpr int kGateFloats = 256;

// Two operands of 64 rows as one of 128: 16 rows of the first, 16 of the second, and so on.  The results of
// either then lie in 16 lanes of each quarter of tensor memory, and all warps have some to read.  The row
// of the first one's row t (the second one's is 16 further on):
__host__ __device__ constexpr int lane_of(int t) { return t / 16 * 32 + t % 16; }
constexpr int kOther = 16;

// A chunk's record: two terms of J and P~ (rows as above), the gates, the third terms.  A piece holds 8 columns
// of all rows, one row after the other: threads that own rows write whole lines, and a product can take either
// the rows or the columns as the contraction.  Pieces 2i and 2i + 1 of the first term are followed by those
// of the second, so that with the columns as rows the two terms' products lie as the two operands do.
constexpr int kRecordGates = 2 * kTermBytes, kRecordThird = kRecordGates + kGateFloats * 4;
constexpr int kRecordBytes = kRecordThird + kTermBytes;
__host__ __device__ constexpr int record_piece(int term, int piece, int row) {
  return (term < 2 ? ((piece / 2) * 4 + term * 2 + piece % 2) * kPieceBytes : kRecordThird + piece * kPieceBytes) + row * 16;
}
enum DeltaGate : int { kEf = 0, kEb = 64, kBeta = 128, kTotal = 192 };  // floats of a record's gates

// Chunk c of sequence i has record slot cu[i] / 64 + i + c: no two chunks share one, and there are
// total / 64 + nseq of them.
__host__ __device__ inline int64_t delta_slots(int64_t total, int64_t nseq) { return total / kDelta + nseq; }

// The chunk of record slot `slot`: rows [row0, row0 + n), number c of the sequence seq with rows [a, b).
struct Chunk {
  int seq, a, b, c, row0, n;
};
// False if the slot has none.  All lanes of a warp.
__device__ __forceinline__ bool find_chunk(const int32_t* cu, int nseq, int total, int64_t slot, int lane, Chunk& x) {
  // the last sequence whose first slot is not above `slot`, 32 candidates at a time
  int64_t lo = 0, hi = nseq;  // it is in [lo, hi)
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool below = i < hi && (i == 0 || min(max(cu[i], 0), total) / kDelta + i <= slot);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  x.seq = static_cast<int>(lo);
  sequence_rows(cu, x.seq, total, x.a, x.b);
  const int64_t c = slot - lo - x.a / kDelta;
  if (c < 0 || c * kDelta >= x.b - x.a) return false;
  x.c = static_cast<int>(c);
  x.row0 = x.a + x.c * kDelta;
  x.n = min(kDelta, x.b - x.row0);
  return true;
}

constexpr int kColumns = 32;                       // columns of V of a chain's CTA
__host__ __device__ inline int delta_tiles(int64_t V) { return static_cast<int>((V + kColumns - 1) / kColumns); }
constexpr int kTermRow = kColumns * 2;             // bytes of a row of one term: 64-byte swizzle

// Descriptor of terms of `kColumns` columns, rows as the contraction; `panel` bytes between terms.
__device__ __forceinline__ uint64_t term_desc(uint32_t addr, uint32_t panel) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) |
         (static_cast<uint64_t>((panel & 0x3FFFFu) >> 4) << 16) |
         (static_cast<uint64_t>((8 * kTermRow) >> 4) << 32) | (1ull << 46) | (4ull << 61);
}
constexpr int kTermStep = 16 * kTermRow / 16;      // descriptor units of 16 rows of a term
// Where the 16-byte piece j of row r of a term lies.
__device__ __forceinline__ uint32_t term_piece(int row, int piece) {
  return static_cast<uint32_t>(row * kTermRow + ((piece ^ ((row >> 1) & 3)) << 4));
}

// Eight fp32 values as bf16 terms of 16 bytes each.
__device__ __forceinline__ void split8(const float* x, uint4 (&out)[kTerms]) {
  const f2 minus = f2_splat(-1.f);
  uint32_t t[kTerms][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2 v = f2_pack(x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int s = 0; s < kTerms; ++s) {
      t[s][i] = f2_to_bf16x2(v);
      if (s + 1 < kTerms) v = f2_fma(bf16x2_to_f2(t[s][i]), minus, v);
    }
  }
#pragma unroll
  for (int s = 0; s < kTerms; ++s) out[s] = make_uint4(t[s][0], t[s][1], t[s][2], t[s][3]);
}

// Contiguous bytes (a multiple of 16, both ends 16-byte aligned) from and to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                   reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}

// The chains' CTAs: 4 warps that move and multiply, 8 that own rows (and 4 that prepare do).
constexpr int kRowWarps = 8;
constexpr int kSlotKq = 2 * kPanelBytes;                // a chunk's K and Q
constexpr int kSlotBytes = kSlotKq + kRecordBytes;      // and its record
constexpr int kStatePanel = 128 * kTermRow, kTokenPanel = kDelta * kTermRow;  // one term
constexpr int kUTile = 2 * kTokenPanel;                 // two terms of u of a chunk, 32 columns

#define DELTA_WAIT(bar, phase) (wait_phase((bar), static_cast<uint32_t>(phase) & 1u))
#define DELTA_WARP_WAIT(bar, phase) (__all_sync(0xffffffffu, DELTA_WAIT(bar, phase)))

// What a row warp has of 16 tokens and 16 columns: tokens lane / 4 and lane / 4 + 8, columns 2 (lane % 4) and the
// next one, and those 8 further on, as pairs [columns][token].
struct Pairs {
  f2 v[2][2];
};
// 16 lanes and 16 columns of tensor memory.
__device__ __forceinline__ void tmem_ld_pairs(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_use8(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(r[i]));
}
// The sum of N groups of kColumns columns, `step` columns apart.
template <int N>
__device__ __forceinline__ Pairs load_sum(uint32_t at, int step = kColumns) {
  uint32_t a[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i) tmem_ld_pairs(at + i * step, a[i]);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) tmem_use8(a[i]);
  Pairs s;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      s.v[j][r] = pair(a[N - 1], 2 * j + r);
#pragma unroll
      for (int i = N - 2; i >= 0; --i) s.v[j][r] = f2_add(s.v[j][r], pair(a[i], 2 * j + r));
    }
  return s;
}
// Pairs of token row `row` (+ 8), columns of half h, to the terms at `base`.
__device__ __forceinline__ void put_pairs(uint32_t base, int row, int h, int lane, const Pairs& p) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t at = base + term_piece(row + 8 * r, 2 * h + j) + (lane & 3) * 4;
      f2 v = p.v[j][r];
#pragma unroll
      for (int s = 0; s < kTerms; ++s) {
        const uint32_t w = f2_to_bf16x2(v);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + s * kTokenPanel), "r"(w) : "memory");
        if (s + 1 < kTerms) v = f2_fma(bf16x2_to_f2(w), f2_splat(-1.f), v);
      }
    }
}
// Four words of each of four neighbouring lanes, turned: lane q gets word q of all (and the other way round).
__device__ __forceinline__ void quad_turn(uint32_t (&w)[4], int lane) {
  const bool odd = lane & 1, high = lane & 2;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[i] : w[i + 1], 1);
    (odd ? w[i] : w[i + 1]) = got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? w[i] : w[i + 2], 2);
    (high ? w[i] : w[i + 2]) = got;
  }
}
// Pairs as bf16, in global memory 16 bytes a lane: lane q of four has token lane / 4 + 8 (q % 2), columns
// 8 (q / 2) on.
__device__ __forceinline__ int quad_token(int lane) { return lane / 4 + 8 * (lane & 1); }
__device__ __forceinline__ int quad_column(int lane) { return 8 * ((lane >> 1) & 1); }
// (Read in words of 4 bytes all the same: turned, they cost the gradient's chain 5 % of its time.)
__device__ __forceinline__ void load_words(const uint16_t* src, int width, int lane, uint32_t (&x)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    x[j] = src && 8 * j < width ? *reinterpret_cast<const uint32_t*>(src + 8 * j + 2 * (lane & 3)) : 0u;
}
__device__ __forceinline__ uint4 quad_words(uint32_t (&w)[4], int lane) {
  quad_turn(w, lane);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Where the gradient's chains keep z: a row warp's pairs, 16 bytes a thread and behind them (kPairsNext) 16 more.
constexpr int kPairsNext = 32;  // ulonglong2
__device__ __forceinline__ int64_t pairs_at(int64_t tile, int row_warp, int lane) {
  return (tile * kRowWarps + row_warp) * 256 + lane * 4;
}

// 16 columns of this thread's row in the terms' groups of kColumns columns: the sum.
__device__ __forceinline__ void load_sum16(uint32_t at, float* x) {
  uint32_t a[kTerms][16];
#pragma unroll
  for (int s = 0; s < kTerms; ++s) tmem_ld16(at + s * kColumns, a[s]);
  tmem_wait_ld();
#pragma unroll
  for (int s = 0; s < kTerms; ++s) tmem_use16(a[s]);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = __uint_as_float(a[kTerms - 1][i]);
#pragma unroll
    for (int s = kTerms - 2; s >= 0; --s) x[i] += __uint_as_float(a[s][i]);
  }
}
// Eight values of row `row` to the terms at `base`.
__device__ __forceinline__ void put_terms8(uint32_t base, uint32_t panel, int row, int piece, const float* x) {
  uint4 t[kTerms];
  split8(x, t);
  const uint32_t at = base + term_piece(row, piece);
#pragma unroll
  for (int s = 0; s < kTerms; ++s) sts128(at + s * panel, t[s].x, t[s].y, t[s].z, t[s].w);
}
__device__ __forceinline__ void unpack8(const uint4& x, float* y) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) cconv::f2_unpack(bf16x2_to_f2(w[j]), y[2 * j], y[2 * j + 1]);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(f2_to_bf16x2(f2_pack(x[0], x[1])), f2_to_bf16x2(f2_pack(x[2], x[3])),
                    f2_to_bf16x2(f2_pack(x[4], x[5])), f2_to_bf16x2(f2_pack(x[6], x[7])));
}

// One chunk's K and Q, 16 tokens a box, `panels` of 64 channels.
__device__ __forceinline__ void load_kq(uint32_t slot, uint32_t bar, const CUtensorMap* mk, const CUtensorMap* mq,
                                        int panels, int hk, int row0) {
  bar_expect(bar, panels * 2 * kSideBytes);
#pragma unroll 1
  for (int j = 0; j < panels; ++j)
#pragma unroll 1
    for (int t = 0; t < kDelta; t += 16) {
      const uint32_t dst = slot + j * kPanelBytes + lane_of(t) * 128;
      load_box(dst, mk, bar, j * kPanelCols, hk, row0 + t);
      load_box(dst + kOther * 128, mq, bar, j * kPanelCols, hk, row0 + t);
    }
}
// Zeroes the rows of tokens n on of a slot's K (and Q): rows of the next sequence must not meet a product over
// the tokens, where 0 * NaN is not 0.  256 threads, i of them this one.
__device__ __forceinline__ void zero_tokens(uint32_t slot, int panels, int n, bool q, int i) {
  const int pieces = (kDelta - n) * 8, sides = q ? 2 : 1;
  for (int e = i; e < panels * sides * pieces; e += 256) {
    const int at = e % pieces, which = e / pieces;
    const int row = lane_of(n + at / 8) + (which % sides) * kOther;
    sts128(slot + which / sides * kPanelBytes + row * 128 + at % 8 * 16, 0, 0, 0, 0);
  }
}

// Descriptors of a record: rows as rows, and columns as rows.
__device__ __forceinline__ uint64_t record_desc(uint32_t addr, bool columns) {
  const uint64_t rows8 = 128 >> 4, piece = kPieceBytes >> 4;
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | ((columns ? rows8 : piece) << 16) |
         ((columns ? piece : rows8) << 32) | (1ull << 46);
}
constexpr int kRecordCols = 4 * kPieceBytes / 16;  // descriptor units of 16 columns, and between the terms
constexpr int kRecordTerm = 2 * kPieceBytes / 16;
constexpr int kRecordRows = 32 * 16 / 16;          // of 16 of an operand's rows
constexpr int kKqRows = 32 * 128 / 16;

// 128 rows of 16 columns, from shared memory to 8 columns of tensor memory: a first operand's k-step.
__device__ __forceinline__ void tmem_copy(uint32_t tmem, uint64_t rows) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;" ::"r"(tmem), "l"(rows) : "memory");
}

// dg_t is the sum of o_i . do_i - v_i . dv_i over the tokens i >= t of the sequence.  Rounding adds up along it,
// so it starts anew at every kAnchorChunks-th chunk, where it is <S_0, D_0>: the chain of the states leaves S_0
// in fp32 there, its way back the product with D, one part from each row warp.  And where e^{g_t} is 0, or the state
// that it acts on (a sequence's first token without an initial state), so is dg_t, the sum behind it, which starts anew
// there too: what rounding left of it is no gradient of a gate that lets nothing through.
constexpr int kAnchorChunks = 8;
constexpr int kAnchorFloats = 128 * kColumns;
// An anchor's place goes by its token: those of a sequence are 512 tokens apart, and the next sequence's first one
// lies as far behind its start.
constexpr int kAnchorTokens = kAnchorChunks * kDelta;
__host__ __device__ inline int64_t delta_anchors(int64_t total) { return total / kAnchorTokens + 1; }
__device__ __forceinline__ int64_t anchor_of(int a, int c) { return a / kAnchorTokens + (a % kAnchorTokens + c * kDelta) / kAnchorTokens; }

__device__ __forceinline__ float dot4(const float4& a, const float4& b) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x)));
}

struct DeltaCall {
  Rows q, k, v, d_o;
  Gates g, beta;          // (beta's values are taken as they are)
  LinearShape s;
  const int32_t* cu;
  Slots slots;
  int checked;            // the verdict on state_indices is there (launch_checks ran)
  int32_t* status;
  float scale;
  const float* initial;
  float* fin;
  uint16_t* o;
  uint8_t* records;       // [slots][Hv] of kRecordBytes
  // the gradient's
  float* z;               // [slots][Hv][tiles] of 64 rows of kColumns, as pairs_at has them
  uint8_t* u;             // [slots][Hv][tiles] two terms of u
  uint8_t *heads, *ends;  // [slots][Hv][tiles] two terms of S_0 and of D
  uint8_t* rest;          // [slots][Hv][tiles] the second term of dv (the first is dv itself)
  float *odots, *vdots, *bdots;  // [2 tiles][Hv][total] parts of o . do, v . dv and dbeta
  uint16_t *dq, *dk, *dv;
  float *dg, *dbeta, *dinit;
  double* sums;           // [Hv][slots] of the chunks' terms of dg, up to the first shut gate
  int* shut;              // [Hv][slots] the last token of the chunk whose gate is shut, or -1
  float *du, *danchors;   // where both chains run at once: du as z, D as the anchors
  float *anchors, *adots; // [anchors][Hv][tiles] states, [anchors][Hv][tiles * kRowWarps] parts of products
};

int launch_delta_prep(const DeltaCall& c, cudaStream_t stream);
int launch_delta_fwd(const DeltaCall& c, cudaStream_t stream);
int launch_delta_states(const DeltaCall& c, cudaStream_t stream);  // the gradient's chain of states
int launch_delta_back(const DeltaCall& c, cudaStream_t stream);    // its chain backwards
int launch_delta_both(const DeltaCall& c, cudaStream_t stream);    // both in one launch
int launch_delta_grads(const DeltaCall& c, cudaStream_t stream);   // dq, dk, dbeta
int launch_delta_gates(const DeltaCall& c, cudaStream_t stream);   // dg, from the chunks' parts and the anchors

}  // namespace cattn
