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

// The chains' CTAs.
constexpr int kChainThreads = 384;  // 4 warps that move and multiply, 8 that own rows
constexpr int kRowWarps = 8;
// a slot of the ring, from a 1024-byte boundary
constexpr int kStageKq = 2 * kPanelBytes;               // panels of 64 rows of K over 64 of Q
constexpr int kStageBytes = kStageKq + kRecordBytes;
constexpr int kStages = 2;
constexpr int kStatePanel = 128 * kTermRow, kTokenPanel = kDelta * kTermRow;  // one term

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

__device__ __forceinline__ void load_bf16x16(const uint16_t* src, int width, bool on, uint4 (&x)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    if (on && 8 * i < width) x[i] = *reinterpret_cast<const uint4*>(src + 8 * i);
  }
}
__device__ __forceinline__ void unpack16(const uint4 (&x)[2], float* y) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) cconv::f2_unpack(bf16x2_to_f2(w[j]), y[8 * i + 2 * j], y[8 * i + 2 * j + 1]);
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
  uint8_t *heads, *ends;  // [slots][Hv][tiles] first terms of S_0 and of D
  float *odots, *vdots, *bdots;  // [2 tiles][Hv][total] parts of o . do, v . dv and dbeta
  uint16_t *dq, *dk, *dv;
  float *dg, *dbeta, *dinit;
};

int launch_delta_prep(const DeltaCall& c, cudaStream_t stream);
int launch_delta_fwd(const DeltaCall& c, cudaStream_t stream);
int launch_delta_states(const DeltaCall& c, cudaStream_t stream);  // the gradient's chain of states
int launch_delta_back(const DeltaCall& c, cudaStream_t stream);    // its chain backwards
int launch_delta_grads(const DeltaCall& c, cudaStream_t stream);   // dq and dk
int launch_delta_gates(const DeltaCall& c, cudaStream_t stream);   // dg and dbeta

}  // namespace cattn
