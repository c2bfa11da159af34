// attn_chunk_host.h -- host interface of the chunked linear-attention kernels.
#pragma once

#include "attn_linear.cuh"

namespace cattn {

// A forward (launch_chunk_fwd), or for the backward the states that ranges hand on and, with q and
// do in k and v, the gradients of states (launch_chunk_states; o is NULL).
struct ChunkCall {
  Rows q, k, v;
  Gates g;
  LinearShape s;
  const int32_t* cu;
  const int32_t* cstart;  // chunk offsets, made by launch_checks; NULL: up to kSmallPlan sequences
  Slots slots;
  const float* initial;
  float* fin;
  int32_t* status;
  float scale;
  uint16_t* o;
  float* carry;  // chunk_fwd_bytes(grid)
  int grid;
  int group;     // CTAs that share a range (forward: 1)
};

struct ChunkBwdCall {
  Rows q, k, v, d_o;
  Gates g;
  LinearShape s;  // total > 0
  const int32_t* cu;
  const int32_t* cstart;
  Slots slots;
  const float* initial;
  float* dinit;
  float scale;
  uint16_t *dq, *dk, *dv;
  float *part_q, *part_k;   // [Hv * tiles][total][K] on 32-byte boundaries, or NULL: one part, or the ring
  float *dots_q, *dots_k;   // [2][Hv * tiles][total]
  float *carry_s, *carry_d; // what launch_chunk_states wrote
  float* ring;              // sum_bytes(grid, K), or NULL: no clusters
  int grid, group;
  bool joined;
};

// Joins the states that ranges hand on (of either direction, or both), where chains are long.
int launch_scan(const ChunkCall& c, float* forward, float* backward, bool* scanned, cudaStream_t stream);
// CTAs of the backward's sweeps that can be resident as clusters of `group`.
int cluster_ctas(int group, int* ctas);
size_t sum_bytes(int grid, int64_t K);
int launch_chunk_bwd(const ChunkBwdCall& c, cudaStream_t stream);
int launch_chunk_fwd(const ChunkCall& c, cudaStream_t stream);
int launch_chunk_states(const ChunkCall& states, const ChunkCall& grads, cudaStream_t stream);
size_t chunk_fwd_bytes(int grid);
int encode_part_map(CUtensorMap* map, float* x, int64_t total, int64_t parts, int64_t C);
int encode_tile_map(CUtensorMap* map, const Rows& x, int64_t total, int64_t H, int64_t C);

}  // namespace cattn
