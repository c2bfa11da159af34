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
// (attn_delta_chain.cu): a CTA takes 32 of them.
//
// Precision: products run on bf16 with fp32 accumulators; an fp32 factor is split into three bf16
// terms (24 bits), and for two such factors the six products of terms down to 2^-16 are summed.
#pragma once

#include "attn_chunk.cuh"

namespace cattn {

constexpr int kDelta = 64;                         // tokens of a chunk
constexpr int kTerms = 3;                          // bf16 terms of an fp32 factor
constexpr int kSideBytes = kDelta * 128;           // 64 rows of a 64-column panel
constexpr int kJpTerm = 128 * 128;                 // one term of J (rows 0..63) over P~ (64..127)
constexpr int kGateFloats = 256;
// a chunk's record: the terms of J and P~ as a product reads them from shared memory, then the gates
constexpr int kRecordBytes = kTerms * kJpTerm + kGateFloats * 4;
enum DeltaGate : int { kEf = 0, kEb = 64, kBeta = 128, kTotal = 192 };  // floats of a record's gates

// Chunk c of sequence i has record slot cu[i] / 64 + i + c: no two chunks share one, and there are
// total / 64 + nseq of them.
__host__ __device__ inline int64_t delta_slots(int64_t total, int64_t nseq) { return total / kDelta + nseq; }

// The sequence and rows of record slot `slot` (rows [row0, row0 + n)); false if it has none.
__device__ __forceinline__ bool find_chunk(const int32_t* cu, int nseq, int total, int64_t slot, int lane,
                                           int& row0, int& n) {
  // the last sequence whose first slot is not above `slot`, 32 candidates at a time
  int64_t lo = 0, hi = nseq;  // it is in [lo, hi)
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
    const bool below = i < hi && (i == 0 || min(max(cu[i], 0), total) / kDelta + i <= slot);
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
    lo += last * step;
    hi = min(hi, lo + step);
  }
  int a, b;
  sequence_rows(cu, static_cast<int>(lo), total, a, b);
  const int64_t c = slot - lo - a / kDelta;
  if (c < 0 || c * kDelta >= b - a) return false;
  row0 = a + static_cast<int>(c) * kDelta;
  n = min(kDelta, b - row0);
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

// Eight fp32 values as three bf16 terms of 16 bytes each.
__device__ __forceinline__ void split8(const float* x, uint4 (&out)[kTerms]) {
  const f2 minus = f2_splat(-1.f);
  uint32_t t[kTerms][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f2 v = f2_pack(x[2 * i], x[2 * i + 1]);
    t[0][i] = f2_to_bf16x2(v);
    v = f2_fma(bf16x2_to_f2(t[0][i]), minus, v);
    t[1][i] = f2_to_bf16x2(v);
    v = f2_fma(bf16x2_to_f2(t[1][i]), minus, v);
    t[2][i] = f2_to_bf16x2(v);
  }
#pragma unroll
  for (int s = 0; s < kTerms; ++s) out[s] = make_uint4(t[s][0], t[s][1], t[s][2], t[s][3]);
}

// Sixteen values of row `row` (column group cg of two) to the three terms at `base`.
__device__ __forceinline__ void put_terms(uint32_t base, uint32_t panel, int row, int cg, const float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 t[kTerms];
    split8(x + 8 * i, t);
    const uint32_t at = base + term_piece(row, cg * 2 + i);
#pragma unroll
    for (int s = 0; s < kTerms; ++s) sts128(at + s * panel, t[s].x, t[s].y, t[s].z, t[s].w);
  }
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

// The chains' CTAs: 4 warps that move and multiply, 8 that own rows of the state and of the tokens,
// 4 that copy first operands to tensor memory and do what the chain does not wait for.
constexpr int kChainThreads = 512;
constexpr int kRowWarps = 8, kCopyWarps = 4;
// the rings: slots of K and Q, then of records, from a 1024-byte boundary
constexpr int kStages = 2;
constexpr int kStageKq = 2 * kPanelBytes;               // panels of 64 rows of K over 64 of Q
constexpr int kOffRecords = kStages * kStageKq;
constexpr int kRingBytes = kOffRecords + kStages * kRecordBytes;
constexpr int kStatePanel = 128 * kTermRow, kTokenPanel = kDelta * kTermRow;  // one term
constexpr int kUTile = 2 * kTokenPanel;                 // two terms of u of a chunk, 32 columns
// columns of tensor memory
constexpr int kTmK = 0, kTmJ = 64, kTmAcc1 = 160, kTmAcc2 = 256, kTmOut1 = 320, kTmOut2 = 384;

#define DELTA_WAIT(bar, phase) (wait_phase((bar), static_cast<uint32_t>(phase) & 1u))
#define DELTA_WARP_WAIT(bar, phase) (__all_sync(0xffffffffu, DELTA_WAIT(bar, phase)))

// The sum of the three terms' products, 16 columns of this thread's row.
__device__ __forceinline__ void load_sum(uint32_t at, float* x) {
  uint32_t a[16], b[16], c[16];
  tmem_ld16(at, a);
  tmem_ld16(at + kColumns, b);
  tmem_ld16(at + 2 * kColumns, c);
  tmem_wait_ld();
  tmem_use16(a);
  tmem_use16(b);
  tmem_use16(c);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(a[i]) + (__uint_as_float(b[i]) + __uint_as_float(c[i]));
}

// Eight columns of products whose accumulators lie in two groups of kColumns: the first terms', and
// the small ones'.
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tmem_use8(uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void load_sum8(uint32_t at, float* x) {
  uint32_t a[8], b[8];
  tmem_ld8(at, a);
  tmem_ld8(at + kColumns, b);
  tmem_wait_ld();
  tmem_use8(a);
  tmem_use8(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(a[i]) + __uint_as_float(b[i]);
}
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

// Row `row` of a 64-column panel (128 bytes, swizzled) to 32 columns of tensor memory; zeros unless `on`.
__device__ __forceinline__ void copy_row(uint32_t tmem, uint32_t panel, int row, bool on) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (on) x = lds128_at(panel + swizzled(row, h * 4 + j));
      w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
    }
    tmem_st16(tmem + 16 * h, w);
  }
}

// One chunk's K and Q (a box of 64 channels and 64 tokens each, `panels` of them) and its record.
__device__ __forceinline__ void load_kq(uint32_t smem, uint32_t bar, const CUtensorMap* mk, const CUtensorMap* mq,
                                        int st, int panels, int hk, int row0) {
  bar_expect(bar, panels * 2 * kSideBytes);
#pragma unroll 1
  for (int j = 0; j < panels; ++j) {
    load_box(smem + st * kStageKq + j * kPanelBytes, mk, bar, j * kPanelCols, hk, row0);
    load_box(smem + st * kStageKq + j * kPanelBytes + kSideBytes, mq, bar, j * kPanelCols, hk, row0);
  }
}
__device__ __forceinline__ void load_record(uint32_t smem, uint32_t bar, const uint8_t* record, int st) {
  bar_expect(bar, kRecordBytes);
  bulk_load(smem + kOffRecords + st * kRecordBytes, record, kRecordBytes, bar);
}

// A (rows of tensor memory at `a`, one term) times three terms of B side by side: the first two as 64
// columns, the third one into the small ones' group.  `steps` of 16 rows of B.
__device__ __forceinline__ void mma_terms(uint32_t acc, uint32_t a, uint64_t b, uint32_t panel, int steps) {
  const uint32_t two = mma_desc(2 * kColumns, false, true), one = mma_desc(kColumns, false, true);
#pragma unroll 1
  for (int j = 0; j < steps; ++j) {
    mma_ts(acc, a + j * 8, b + j * kTermStep, two, j > 0);
    mma_ts(acc + kColumns, a + j * 8, b + (2 * panel >> 4) + j * kTermStep, one, true);
  }
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
  float* z;               // [total][Hv][V]
  uint8_t* u;             // [slots][Hv][tiles] two terms of u
  uint8_t *heads, *ends;  // [slots][Hv][tiles] first terms of S_0 and of D
  float *odots, *vdots, *bdots;  // [tiles][Hv][total] parts of o . do, v . dv and dbeta
  uint16_t *dq, *dk, *dv;
  float *dg, *dbeta, *dinit;
  double* sums;           // [Hv][slots] of the chunks' terms of dg
};

int launch_delta_prep(const DeltaCall& c, cudaStream_t stream);
int launch_delta_fwd(const DeltaCall& c, cudaStream_t stream);
int launch_delta_states(const DeltaCall& c, cudaStream_t stream);  // the gradient's chain of states
int launch_delta_back(const DeltaCall& c, cudaStream_t stream);    // its chain backwards
int launch_delta_grads(const DeltaCall& c, cudaStream_t stream);   // dq, dk, dbeta
int launch_delta_gates(const DeltaCall& c, cudaStream_t stream);   // dg, from the chunks' parts

}  // namespace cattn
