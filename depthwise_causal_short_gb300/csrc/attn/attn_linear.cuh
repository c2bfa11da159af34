// attn_linear.cuh -- arguments shared by the linear-attention kernels.
#pragma once

#include "attn.cuh"

namespace cattn {

// A [total, H, C] bf16 tensor.
struct Rows {
  const uint16_t* p;
  int64_t st, sh;
};

struct Gates {
  const float* p;
  int64_t st, sh;
  __device__ __forceinline__ float at(int64_t t, int h) const {
    return clamp_decay(__ldg(p + t * st + h * sh));
  }
};

struct LinearShape {
  int total, Hk, Hv, K, V, nseq;
};

// State slot of sequence i, or -1 if it has none that can be used.
struct Slots {
  const int32_t* idx;
  int64_t S;
  __device__ __forceinline__ int64_t of(int i) const {
    if (!idx) return i;
    const int s = idx[i];
    return s >= 0 && s < S ? s : -1;
  }
};

// Checks of the entry points' arguments: a cconv_status.
int check_gates(const float* g, int64_t rows, int64_t H, int64_t st, int64_t sh);
int check_linear(const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh,
                 const void* v, int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh,
                 int64_t rows, int64_t Hk, int64_t Hv, int64_t K, int64_t V, const void* o);
int check_states(const int32_t* cu, int64_t nseq, int64_t Hv, const float* initial, const float* fin,
                 const int32_t* idx, int64_t S, int32_t* status);
int check_sizes(int64_t total, int64_t nseq, int64_t Hk, int64_t Hv, int64_t K, int64_t V);

}  // namespace cattn
