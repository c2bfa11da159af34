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

}  // namespace cattn
