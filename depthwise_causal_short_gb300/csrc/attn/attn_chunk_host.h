// attn_chunk_host.h -- host interface of the chunked linear-attention kernels.
#pragma once

#include "attn_linear.cuh"

namespace cattn {

struct ChunkCall {
  Rows q, k, v;
  Gates g;
  LinearShape s;
  const int32_t* cu;
  const int32_t* cstart;  // chunk offsets, made by launch_checks
  Slots slots;
  const float* initial;
  float* fin;
  const int32_t* status;
  float scale;
  uint16_t* o;
  float* carry;  // chunk_fwd_bytes(grid)
  int grid;
};

int launch_chunk_fwd(const ChunkCall& c, cudaStream_t stream);
size_t chunk_fwd_bytes(int grid);
int encode_tile_map(CUtensorMap* map, const Rows& x, int64_t total, int64_t H, int64_t C);

}  // namespace cattn
