// attn.cuh -- what the mixer kernels of libcattn share, on top of the convolution's helpers.
#pragma once

#include "../common.cuh"
#include "../../../include/cattn.h"

namespace cattn {

using cconv::launch_pdl;
using cconv::report_cuda;

enum FaultCode : unsigned {
  kFaultWait = 1u,      // a bounded wait ran out
  kFaultSeqlens = 4u,   // an ill-formed cu_seqlens was passed
  kFaultPosition = 8u,  // a position outside the rotation tables
};

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 16;
constexpr int kMaxK = 128;
constexpr int kMaxV = 256;

// Each translation unit owns a device fault word and registers a reader of it.
struct FaultReader {
  explicit FaultReader(int (*read)(unsigned*));
};

int bind_context();
int sm_count(int* sms);

__host__ __device__ inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A [total, H, C] bf16 activation with strides (st, sh): the rules of cattn.h.
inline int check_rows(const void* p, int64_t total, int64_t H, int64_t st, int64_t sh) {
  if (!aligned(p, 16)) return CCONV_ERR_ALIGN;
  if (total > 1) {
    if (st < 1) return CCONV_ERR_STRIDE;
    if (st % 8 != 0) return CCONV_ERR_ALIGN;
  }
  if (H > 1) {
    if (sh < 1) return CCONV_ERR_STRIDE;
    if (sh % 8 != 0) return CCONV_ERR_ALIGN;
  }
  return CCONV_OK;
}

// Rows [a, b) of sequence i, inside [0, total] whatever cu_seqlens holds.
__device__ __forceinline__ void sequence_rows(const int32_t* cu, int i, int total, int& a, int& b) {
  a = min(max(cu[i], 0), total);
  b = min(max(cu[i + 1], a), total);
}

__device__ __forceinline__ float clamp_decay(float g) { return g < -128.f ? -128.f : g; }

// The offences of up to 32 state indices, one a lane (s: the lane's, -1 among them with pad).
// Every lane of the warp gets the union.
__device__ __forceinline__ unsigned check_indices(int s, int n, int64_t S, bool pad, int lane) {
  unsigned bad = 0;
  const bool live = lane < n && !(pad && s == -1);
  if (live && s < 0) bad = CCONV_IDX_NEGATIVE;
  if (live && s >= S) bad = CCONV_IDX_OUT_OF_RANGE;
  const bool slot = live && bad == 0;
  // lanes without a usable slot get values of their own
  const unsigned same = __match_any_sync(0xffffffffu, slot ? s : -2 - lane);
  if (slot && (same & (same - 1))) bad = CCONV_IDX_DUPLICATE;
  return __reduce_or_sync(0xffffffffu, bad);
}

// Checks n state indices against S slots (negative, >= S, repeated; -1 allowed with pad), and
// nseq + 1 row offsets when cu is given; writes status[0..1] when idx is given, and with
// `cstart` the offsets of the sequences' 128-token chunks (an empty sequence has one; all zero
// for ill-formed offsets).  One CTA.
int launch_checks(const int32_t* idx, int64_t n, int64_t S, int pad, int32_t* status,
                  const int32_t* cu, int64_t nseq, int64_t total, int32_t* cstart,
                  cudaStream_t stream);

}  // namespace cattn
