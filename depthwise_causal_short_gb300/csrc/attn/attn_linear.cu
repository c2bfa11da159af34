// attn_linear.cu -- linear attention with a decay for each token and head over packed
// sequences: the entry points, and the sums that finish the backward.
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale q_t^T S_t
//   D_t = scale q_t do_t^T + e^{g_{t+1}} D_{t+1}
//   dq_t = scale S_t do_t,  dk_t = D_t v_t,  dv_t = D_t^T k_t
//
// and dg_t = sum over i >= t of (q_i . dq'_i - k_i . dk'_i), where dq' and dk' leave out the
// token's own product with itself: a change of g_t moves every pair (i, j) with j < t <= i,
// and q_i . dq'_i sums the pairs j < i that end at i, k_j . dk'_j the pairs i > j that start at
// j.  (With the products i = j in both sums they would cancel only to rounding, and drown the
// dg of heads that forget fast.)
#include "attn_chunk.cuh"
#include "attn_chunk_host.h"

namespace cattn {

constexpr int64_t kMaxSeqs = int64_t(1) << 30;
constexpr int64_t kMaxGroup = 8;    // CTAs of a cluster
constexpr int64_t kSmallSeqs = 32;  // kSmallPlan: the kernels plan for themselves

// dst[t, hk, :] = sum over the (value head, column tile) parts of key head hk, in their order.
// A thread takes 8 channels of one row; bound by memory (4 bytes a part, 2 out): 32 us, 5.3 TB/s, for
// 2 parts of 16384 rows of 8 heads of 128.
__global__ void __launch_bounds__(256)
    cattn_linear_heads_kernel(const float* part, int total, int Hk, int K, int parts, uint16_t* dst) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int pieces = K / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(total) * Hk * pieces) return;
  const int piece = static_cast<int>(i % pieces);
  const int hk = static_cast<int>(i / pieces % Hk);
  const int64_t t = i / pieces / Hk;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll 4
  for (int j = 0; j < parts; ++j) {
    const float4* src = reinterpret_cast<const float4*>(
        part + ((static_cast<int64_t>(hk) * parts + j) * total + t) * K + piece * 8);
    const float4 x = __ldcs(src), y = __ldcs(src + 1);
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    b.x += y.x, b.y += y.y, b.z += y.z, b.w += y.w;
  }
  using cconv::f2_pack;
  using cconv::f2_to_bf16x2;
  *reinterpret_cast<uint4*>(dst + (t * Hk + hk) * K + piece * 8) =
      make_uint4(f2_to_bf16x2(f2_pack(a.x, a.y)), f2_to_bf16x2(f2_pack(a.z, a.w)),
                 f2_to_bf16x2(f2_pack(b.x, b.y)), f2_to_bf16x2(f2_pack(b.z, b.w)));
}

// dg of one sequence and value head, from the rows' sums x_i = qdot_i - kdot_i:
//   dg_t = dg_b + sum of x_i over t <= i < b
// between the anchors a <= t < b: the starts of the ranges that lie in the sequence (where
// dg_a = scale <D, S> is known from the whole states), the sequence's end (0), and its start
// (0 without an initial state; with one not known).  What the sum to a misses of dg_a, rounding
// of the x_i, is spread evenly over the tokens between.  One CTA for each stretch between anchors:
// the first `grid` ones for those that begin at their range's start, the others for those that
// begin at a sequence's; a launch for each column tile of V, the second of which adds.  A stretch
// is cut into a part for each warp, whose sums meet in shared memory before the running ones are
// made (a warp a stretch, with 8 stretches in a CTA, took 22 us of 16384 rows and 16 heads where
// this takes 10).
constexpr int kDgThreads = 256, kDgPer = 4, kDgWarps = kDgThreads / 32;
constexpr int kSlices = 2;  // parts of a unit's dots

struct DgArgs {
  Plan plan;
  const float *qdot, *kdot;  // [kSlices][heads * tiles][total]
  const float* anchors;      // [grid][4]
  int grid, open, tile;      // CTAs of the sweeps; whether the sequences have initial states
  float* dg;
};

// Stretch `at`, by the whole CTA; `sums`: a float a warp.
__device__ __forceinline__ void dg_stretch(const DgArgs& p, const Plan& plan, int nch, int64_t units,
                                           int64_t at, float* sums) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t ranges = range_count(plan, p.grid, units);
  const bool inside = at < p.grid;  // it begins at a range's start
  int64_t u, range = 0;  // its first unit, and the range that this is in
  Walker w;
  if (inside) {
    range = at / plan.group;
    if (range >= ranges) return;
    u = units * range / ranges;
    w.seek(&plan, nch, u, static_cast<int>(at % plan.group));
    if (w.first() || w.ht % plan.tiles != p.tile) return;
  } else {
    const int seq = static_cast<int>((at - p.grid) / plan.heads);
    const int ht = static_cast<int>((at - p.grid) % plan.heads) * plan.tiles + p.tile;
    u = static_cast<int64_t>(ht / plan.group) * nch + plan.cstart[seq];
    w.seek(&plan, nch, u, ht % plan.group);
    range = u * ranges / units;
    while (units * range / ranges > u) --range;
    while (units * (range + 1) / ranges <= u) ++range;
  }
  const int h = w.ht / plan.tiles, member = w.ht % plan.group;
  auto anchor = [&](int64_t i) {
    const float* a = p.anchors + 4 * (i * plan.group + member);
    return (a[0] + a[1]) + (a[2] + a[3]);
  };
  const int64_t end = u - w.c + w.ce, stop = units * (range + 1) / ranges;
  const bool reaches = stop >= end;  // the sequence's end
  const int left = w.row0();
  const int right = reaches ? w.base + w.len : left + static_cast<int>(stop - u) * kChunk;
  if (right <= left) return;
  const float known = reaches ? 0.f : anchor(range + 1);  // dg at `right`
  const bool tied = inside || !p.open;

  const int64_t slice = static_cast<int64_t>(plan.heads) * plan.tiles * plan.total;
  const float* q = p.qdot + static_cast<int64_t>(w.ht) * plan.total;
  const float* k = p.kdot + static_cast<int64_t>(w.ht) * plan.total;
  constexpr int kStep = 32 * kDgPer;
  // this warp's tokens [from, to): whole steps, from the right end on
  const int each = ((right - left + kStep - 1) / kStep + kDgWarps - 1) / kDgWarps * kStep;
  const int to = max(left, right - warp * each), from = max(left, to - each);
  // x of this lane's tokens top, top - 1, .., summed up one after the other
  auto load = [&](int top, float* x) {
#pragma unroll
    for (int j = 0; j < kDgPer; ++j) x[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i)
#pragma unroll
      for (int j = 0; j < kDgPer; ++j)
        if (top - j >= from) x[j] += q[i * slice + top - j] - k[i * slice + top - j];
#pragma unroll
    for (int j = 1; j < kDgPer; ++j) x[j] += x[j - 1];
  };
  float x[kDgPer], total = 0.f;
  for (int hi = to; hi > from; hi -= kStep) {
    load(hi - 1 - lane * kDgPer, x);
    total += x[kDgPer - 1];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  float carry = known, all = known;
#pragma unroll
  for (int i = 0; i < kDgWarps; ++i) {
    if (i < warp) carry += sums[i];
    all += sums[i];
  }
  const float miss = tied ? ((inside ? anchor(range) : 0.f) - all) / static_cast<float>(right - left) : 0.f;
  for (int hi = to; hi > from; hi -= kStep) {
    const int top = hi - 1 - lane * kDgPer;
    load(top, x);
    float run = x[kDgPer - 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += y;
    }
    float before = __shfl_up_sync(0xffffffffu, run, 1);  // the lanes before this one
    before = lane > 0 ? carry + before : carry;
    carry += __shfl_sync(0xffffffffu, run, 31);
#pragma unroll
    for (int j = 0; j < kDgPer; ++j)
      if (top - j >= from) {
        const float v = before + x[j] + miss * static_cast<float>(right - (top - j));
        float* dst = p.dg + static_cast<int64_t>(top - j) * plan.heads + h;
        *dst = p.tile ? *dst + v : v;
      }
  }
}

__global__ void __launch_bounds__(kDgThreads) cattn_linear_dg_kernel(const __grid_constant__ DgArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ SmallPlan small;
  __shared__ float sums[kDgWarps];
  Plan plan = p.plan;
  if (plan.small) small_plan(plan, small, false, nullptr);
  int nch;
  const int64_t units = unit_count(plan, nch);
  if (units == 0) return;
  const int64_t count = p.grid + static_cast<int64_t>(plan.nseq) * plan.heads;
  for (int64_t at = blockIdx.x; at < count; at += gridDim.x) {
    dg_stretch(p, plan, nch, units, at, sums);
    __syncthreads();  // (whole CTAs leave a stretch early)
  }
}

static int check_gates(const float* g, int64_t rows, int64_t H, int64_t st, int64_t sh) {
  if (!g) return CCONV_ERR_NULL;
  if (!aligned(g, 4)) return CCONV_ERR_ALIGN;
  if ((rows > 1 && st < 0) || (H > 1 && sh < 0)) return CCONV_ERR_STRIDE;
  return CCONV_OK;
}

int check_linear(const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh,
                 const void* v, int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh,
                 int64_t rows, int64_t Hk, int64_t Hv, int64_t K, int64_t V, const void* o) {
  if (rows < 0 || rows > kMaxRows || Hk < 1 || Hv < 1 || Hv > 65535 || Hv % Hk != 0 || K < 8 ||
      K > kMaxK || V < 8 || V > kMaxV)
    return CCONV_ERR_SHAPE;
  if (K % 8 != 0 || V % 8 != 0) return CCONV_ERR_ALIGN;
  if (rows == 0) return CCONV_OK;
  if (!q || !k || !v || !o) return CCONV_ERR_NULL;
  int rc = check_gates(g, rows, Hv, sgt, sgh);
  if (rc == CCONV_OK) rc = check_rows(q, rows, Hk, sqt, sqh);
  if (rc == CCONV_OK) rc = check_rows(k, rows, Hk, skt, skh);
  if (rc == CCONV_OK) rc = check_rows(v, rows, Hv, svt, svh);
  if (rc != CCONV_OK) return rc;
  return aligned(o, 16) ? CCONV_OK : CCONV_ERR_ALIGN;
}

static int check_states(const int32_t* cu, int64_t nseq, int64_t Hv, const float* initial, const float* fin,
                        const int32_t* idx, int64_t S, int32_t* status) {
  if (!cu) return CCONV_ERR_NULL;
  if (nseq < 1 || nseq > kMaxSeqs || nseq * Hv > (int64_t(1) << 31) - 1) return CCONV_ERR_SHAPE;
  if (!aligned(cu, 4)) return CCONV_ERR_ALIGN;
  if (idx) {
    if (!status) return CCONV_ERR_NULL;
    if (S < 1 || S > CCONV_UPDATE_MAX_SLOTS) return CCONV_ERR_SHAPE;
    if (!aligned(idx, 4) || !aligned(status, 4)) return CCONV_ERR_ALIGN;
  } else if ((initial || fin) && S < nseq) {
    return CCONV_ERR_SHAPE;
  }
  return aligned(initial, 32) && aligned(fin, 32) ? CCONV_OK : CCONV_ERR_ALIGN;
}

static LinearShape shape_of(int64_t total, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                            int64_t nseq) {
  return LinearShape{static_cast<int>(total), static_cast<int>(Hk), static_cast<int>(Hv),
                     static_cast<int>(K), static_cast<int>(V), static_cast<int>(nseq)};
}

static Rows rows(const void* p, int64_t st, int64_t sh) {
  return Rows{static_cast<const uint16_t*>(p), st, sh};
}

// CTAs of the chunked kernels: one per SM, or one per unit where there can be no more units.
static int chunk_grid(int64_t total, int64_t nseq, int64_t Hv, int64_t V, int* grid) {
  int sms = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  const int64_t units = Hv * ((V + 127) / 128) * (total / 128 + nseq);
  *grid = static_cast<int>(units < sms ? units : sms);
  return CCONV_OK;
}

// CTAs of the backward, and how many share a range: the members of a key head (its value heads
// and their column tiles) as a cluster, where these are even and at most 8.  Measured on 16384 rows
// with heads of 128, clusters against sums through memory, us: 2 members 381 / 447, 4 members
// 379 / 443 (V of 256: 395 / 470), 6 members 332 / 350, 8 members 416 / 449, but 3 members 398 / 350,
// 5 353 / 300, 7 448 / 396: a share of an odd number of 8-column pieces is half as fast to add up and
// to store, and all members wait for the slowest.
static int bwd_grid(int64_t total, int64_t nseq, int64_t Hk, int64_t Hv, int64_t V, int* grid,
                    int* group) {
  *group = 1;
  if (chunk_grid(total, nseq, Hv, V, grid) != CCONV_OK) return CCONV_ERR_CUDA;
  const int64_t tiles = (V + 127) / 128, members = Hv / Hk * tiles;
  if (members % 2 != 0 || members > kMaxGroup) return CCONV_OK;
  int ctas = 0;
  if (cluster_ctas(static_cast<int>(members), &ctas) != CCONV_OK) return CCONV_ERR_CUDA;
  if (ctas < members) return CCONV_OK;
  const int64_t ranges = Hk * (total / 128 + nseq), most = ctas / members;
  *group = static_cast<int>(members);
  *grid = static_cast<int>(members * (ranges < most ? ranges : most));
  return CCONV_OK;
}

// The chunk offsets at the head of the workspace.
static size_t offsets_bytes(int64_t nseq) { return (static_cast<size_t>(nseq + 1) * 4 + 15) / 16 * 16; }

// What a backward call keeps in its workspace, from a 256-byte boundary.
struct BwdWork {
  size_t offsets, carry_s, carry_d, dots_q, dots_k, part_q, part_k, ring, bytes;
};
static BwdWork bwd_work(int64_t total, int64_t nseq, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                        int grid, int group) {
  const size_t tiles = static_cast<size_t>((V + 127) / 128), heads = static_cast<size_t>(Hv) * tiles;
  const bool parts = group == 1 && heads > static_cast<size_t>(Hk);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += (n + 255) / 256 * 256;
    return r;
  };
  BwdWork w{};
  w.offsets = take(offsets_bytes(nseq));
  w.carry_s = take(chunk_fwd_bytes(grid));
  w.carry_d = take(chunk_fwd_bytes(grid));
  w.dots_q = take(kSlices * heads * static_cast<size_t>(total) * 4);
  w.dots_k = take(kSlices * heads * static_cast<size_t>(total) * 4);
  w.part_q = take(parts ? heads * static_cast<size_t>(total) * K * 4 : 0);
  w.part_k = take(parts ? heads * static_cast<size_t>(total) * K * 4 : 0);
  w.ring = take(group > 1 ? sum_bytes(grid, K) : 0);
  w.bytes = at + 256;
  return w;
}

static int check_sizes(int64_t total, int64_t nseq, int64_t Hk, int64_t Hv, int64_t K, int64_t V) {
  if (total < 0 || total > kMaxRows || nseq < 1 || nseq > kMaxSeqs || Hk < 1 ||
      Hv < 1 || Hv > 65535 || Hv % Hk != 0 || K < 8 || K > kMaxK || V < 8 || V > kMaxV)
    return CCONV_ERR_SHAPE;
  return CCONV_OK;
}

}  // namespace cattn

extern "C" CCONV_API int cattn_linear_fwd_workspace_bytes(int64_t total, int64_t nseq, int64_t Hk,
                                                          int64_t Hv, int64_t K, int64_t V,
                                                          size_t* bytes) {
  using namespace cattn;
  if (!bytes) return CCONV_ERR_NULL;
  const int rc = check_sizes(total, nseq, Hk, Hv, K, V);
  int grid = 0;
  if (rc != CCONV_OK) return rc;
  if (chunk_grid(total, nseq, Hv, V, &grid) != CCONV_OK) return CCONV_ERR_CUDA;
  *bytes = offsets_bytes(nseq) + chunk_fwd_bytes(grid);
  return CCONV_OK;
}

extern "C" CCONV_API int cattn_linear_bwd_workspace_bytes(int64_t total, int64_t nseq, int64_t Hk,
                                                          int64_t Hv, int64_t K, int64_t V,
                                                          size_t* bytes) {
  using namespace cattn;
  if (!bytes) return CCONV_ERR_NULL;
  const int rc = check_sizes(total, nseq, Hk, Hv, K, V);
  int grid = 0, group = 1;
  if (rc != CCONV_OK) return rc;
  if (bwd_grid(total, nseq, Hk, Hv, V, &grid, &group) != CCONV_OK) return CCONV_ERR_CUDA;
  *bytes = bwd_work(total, nseq, Hk, Hv, K, V, grid, group).bytes;
  return CCONV_OK;
}

extern "C" CCONV_API int cattn_linear_fwd(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
    int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh, int64_t total, int64_t Hk,
    int64_t Hv, int64_t K, int64_t V, const int32_t* cu_seqlens, int64_t nseq, float scale,
    const float* initial_state, float* final_state, const int32_t* state_indices, int64_t S,
    int32_t* status_dev, void* o, void* workspace, size_t workspace_bytes, cconv_stream_t stream) {
  using namespace cattn;
  int rc = check_linear(q, sqt, sqh, k, skt, skh, v, svt, svh, g, sgt, sgh, total, Hk, Hv, K, V, o);
  if (rc == CCONV_OK)
    rc = check_states(cu_seqlens, nseq, Hv, initial_state, final_state, state_indices, S, status_dev);
  if (rc != CCONV_OK) return rc;
  int grid = 0;
  if (chunk_grid(total, nseq, Hv, V, &grid) != CCONV_OK) return CCONV_ERR_CUDA;
  if (!workspace || workspace_bytes < offsets_bytes(nseq) + chunk_fwd_bytes(grid))
    return CCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
  int32_t* cstart = nseq > kSmallSeqs ? static_cast<int32_t*>(workspace) : nullptr;
  if (cstart) {
    rc = launch_checks(state_indices, nseq, S, 0, status_dev, cu_seqlens, nseq, total, cstart, stream);
    if (rc != CCONV_OK) return rc;
  }
  ChunkCall c{};
  c.q = rows(q, sqt, sqh), c.k = rows(k, skt, skh), c.v = rows(v, svt, svh);
  c.g = Gates{g, sgt, sgh};
  c.s = shape_of(total, Hk, Hv, K, V, nseq);
  c.cu = cu_seqlens, c.cstart = cstart;
  c.slots = Slots{state_indices, S};
  c.initial = initial_state, c.fin = final_state;
  c.status = status_dev;
  c.scale = scale;
  c.o = static_cast<uint16_t*>(o);
  c.carry = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + offsets_bytes(nseq));
  c.grid = grid, c.group = 1;
  return launch_chunk_fwd(c, stream);
}

extern "C" CCONV_API int cattn_linear_bwd(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
    int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh, const void* do_, int64_t sot,
    int64_t soh, int64_t total, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
    const int32_t* cu_seqlens, int64_t nseq, float scale, const float* initial_state,
    const int32_t* state_indices, int64_t S, int32_t* status_dev, void* dq, void* dk, void* dv,
    float* dg, float* d_initial_state, void* workspace, size_t workspace_bytes,
    cconv_stream_t stream) {
  using namespace cattn;
  int rc = check_linear(q, sqt, sqh, k, skt, skh, v, svt, svh, g, sgt, sgh, total, Hk, Hv, K, V, dv);
  if (rc == CCONV_OK)
    rc = check_states(cu_seqlens, nseq, Hv, initial_state, nullptr, state_indices, S, status_dev);
  if (rc != CCONV_OK) return rc;
  if (!aligned(d_initial_state, 32)) return CCONV_ERR_ALIGN;
  if (total > 0) {
    if (!do_ || !dq || !dk || !dg) return CCONV_ERR_NULL;
    rc = check_rows(do_, total, Hv, sot, soh);
    if (rc != CCONV_OK) return rc;
    if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dg, 16)) return CCONV_ERR_ALIGN;
  }
  int grid = 0, group = 1;
  if (bwd_grid(total, nseq, Hk, Hv, V, &grid, &group) != CCONV_OK) return CCONV_ERR_CUDA;
  const BwdWork w = bwd_work(total, nseq, Hk, Hv, K, V, grid, group);
  if (total > 0) {
    if (!workspace || workspace_bytes < w.bytes) return CCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
  }
  uint8_t* ws = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
  int32_t* cstart =
      total > 0 && nseq > kSmallSeqs ? reinterpret_cast<int32_t*>(ws + w.offsets) : nullptr;
  if (cstart || total == 0) {
    rc = launch_checks(state_indices, nseq, S, 0, status_dev, cu_seqlens, nseq, total, cstart, stream);
    if (rc != CCONV_OK) return rc;
  }
  if (total == 0) {
    if (d_initial_state && !cconv::recording_launches() &&
        report_cuda("cudaMemsetAsync",
                    cudaMemsetAsync(d_initial_state, 0, static_cast<size_t>(nseq) * Hv * K * V * 4,
                                    stream)) != cudaSuccess)
      return CCONV_ERR_CUDA;
    return CCONV_OK;
  }

  ChunkCall states{};
  states.q = rows(q, sqt, sqh), states.k = rows(k, skt, skh), states.v = rows(v, svt, svh);
  states.g = Gates{g, sgt, sgh};
  states.s = shape_of(total, Hk, Hv, K, V, nseq);
  states.cu = cu_seqlens, states.cstart = cstart;
  states.slots = Slots{state_indices, S};
  states.initial = initial_state;
  states.status = status_dev;
  states.grid = grid, states.group = group;
  states.carry = reinterpret_cast<float*>(ws + w.carry_s);
  ChunkCall grads = states;
  grads.k = states.q, grads.v = rows(do_, sot, soh);
  grads.initial = nullptr;
  grads.carry = reinterpret_cast<float*>(ws + w.carry_d);
  rc = launch_chunk_states(states, grads, stream);
  if (rc != CCONV_OK) return rc;

  bool joined = false;
  rc = launch_scan(states, states.carry, grads.carry, &joined, stream);
  if (rc != CCONV_OK) return rc;

  ChunkBwdCall c{};
  c.joined = joined;
  c.q = states.q, c.k = states.k, c.v = states.v, c.d_o = grads.v;
  c.g = states.g, c.s = states.s, c.cu = cu_seqlens, c.cstart = cstart, c.slots = states.slots;
  c.initial = initial_state, c.dinit = d_initial_state, c.scale = scale;
  c.dq = static_cast<uint16_t*>(dq), c.dk = static_cast<uint16_t*>(dk);
  c.dv = static_cast<uint16_t*>(dv);
  const int tiles = static_cast<int>((V + 127) / 128), parts = static_cast<int>(Hv / Hk) * tiles;
  if (group > 1) {
    c.ring = reinterpret_cast<float*>(ws + w.ring);
  } else if (parts > 1) {
    c.part_q = reinterpret_cast<float*>(ws + w.part_q);
    c.part_k = reinterpret_cast<float*>(ws + w.part_k);
  }
  c.dots_q = reinterpret_cast<float*>(ws + w.dots_q);
  c.dots_k = reinterpret_cast<float*>(ws + w.dots_k);
  c.carry_s = states.carry, c.carry_d = grads.carry;
  c.grid = grid, c.group = group;
  rc = launch_chunk_bwd(c, stream);
  if (rc != CCONV_OK) return rc;

  if (c.part_q) {
    const unsigned ctas = static_cast<unsigned>((total * Hk * (K / 8) + 255) / 256);
    for (int side = 0; side < 2; ++side)
      if (launch_pdl(cattn_linear_heads_kernel, dim3(ctas), dim3(256), 0, stream,
                     static_cast<const float*>(side ? c.part_k : c.part_q), c.s.total, c.s.Hk, c.s.K,
                     parts, side ? c.dk : c.dq) != cudaSuccess)
        return CCONV_ERR_CUDA;
  }
  DgArgs d{};
  d.plan = Plan{cu_seqlens, cstart, c.s.nseq, tiles, c.s.Hv, group, cstart == nullptr, c.s.total, nullptr, 0, nullptr};
  d.qdot = c.dots_q, d.kdot = c.dots_k;
  d.anchors = c.carry_d + static_cast<int64_t>(grid) * kStateFloats;
  d.grid = grid, d.open = initial_state != nullptr;
  d.dg = dg;
  const int64_t stretches = grid + nseq * Hv, most = 1 << 20;
  for (d.tile = 0; d.tile < tiles; ++d.tile)
    if (launch_pdl(cattn_linear_dg_kernel, dim3(static_cast<unsigned>(stretches < most ? stretches : most)),
                   dim3(kDgThreads), 0, stream, d) != cudaSuccess)
      return CCONV_ERR_CUDA;
  return CCONV_OK;
}
