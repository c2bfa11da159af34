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

constexpr int kColumns = 32;                       // columns of V of a chain's CTA
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
};

int launch_delta_prep(const DeltaCall& c, cudaStream_t stream);
int launch_delta_fwd(const DeltaCall& c, cudaStream_t stream);

}  // namespace cattn
