// attn_linear.cu -- linear attention with a decay for each token and head over packed
// sequences: the entry points and the recurrence.
//
// One sweep gives all four products: with roles (a, b, c),
//
//   M <- e^{g} M + b_t c_t^T,   out_t = M^T a_t        M: [A, C], A = |a| = |b|, C = |c|
//
//   o  : a = q,  b = k,  c = v   forwards   (M = S)
//   dq : a = do, b = v,  c = k   forwards   (M = S^T)
//   dk : a = v,  b = do, c = q   backwards  (M = D^T)
//   dv : a = k,  b = q,  c = do  backwards  (M = D)
//
// and dg_t = sum over i >= t of (q_i . dq'_i - k_i . dk'_i), where dq' and dk' leave out the
// token's own product with itself: a change of g_t moves every pair (i, j) with j < t <= i,
// and q_i . dq'_i sums the pairs j < i that end at i, k_j . dk'_j the pairs i > j that start at
// j.  (With the products i = j in both sums they would cancel only to rounding, and drown the
// dg of heads that forget fast.)
#include "attn_chunk_host.h"

namespace cattn {

using cconv::bf16_to_f32;

constexpr int kCols = 32;   // columns of M in one CTA (one a lane)
constexpr int kWarps = 4;   // rows of M are dealt out to the warps
constexpr int kTile = 16;   // tokens staged at once
constexpr int64_t kMaxSeqs = int64_t(1) << 30;

struct SweepArgs {
  Rows a, b, c;
  Gates g;
  int ha, hb, hc;        // heads of a, b, c (value heads map onto them)
  int A, C;
  LinearShape s;
  const int32_t* cu;
  Slots slots;
  const float* m0;       // [S, Hv, K, V] or NULL
  float* m1;             // written at the end of each sequence, or NULL
  const int32_t* status; // states are written only if status is NULL or [0] == CCONV_OK
  bool m1_slots;         // m1's slot is the sequence's state slot (else the sequence)
  bool transposed;       // M is S^T: m0 and m1 are [C, A] in memory
  float m1_scale;
  float scale;
  uint16_t* out;         // [total, Hv, C] bf16, or
  float* out32;          // the same in fp32, and
  Rows x;                // with it the dots of x (c's heads) and out without the token's own
  float* dots;           // product, of this CTA's columns: [slice, total, Hv]
};

// One CTA: one sequence, one value head, kCols columns.
template <int ROWS, bool REVERSE>
__global__ void __launch_bounds__(kWarps * 32) cattn_linear_sweep_kernel(SweepArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float sa[kTile][kWarps * ROWS], sb[kTile][kWarps * ROWS];
  __shared__ float part[kTile][kWarps][kCols], own[kTile][kWarps];
  __shared__ float decay[kTile];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int slices = (p.C + kCols - 1) / kCols;
  const int64_t cta = blockIdx.x;
  const int slice = static_cast<int>(cta % slices);
  const int h = static_cast<int>(cta / slices % p.s.Hv);
  const int seq = static_cast<int>(cta / slices / p.s.Hv);
  const int col = slice * kCols + lane;
  const bool on = col < p.C;
  int t0, t1;
  sequence_rows(p.cu, seq, p.s.total, t0, t1);
  const int ha = h / (p.s.Hv / p.ha), hb = h / (p.s.Hv / p.hb), hc = h / (p.s.Hv / p.hc);
  const int64_t slot = p.slots.of(seq);
  const int64_t head = static_cast<int64_t>(p.A) * p.C;

  float m[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int row = warp * ROWS + r;
    m[r] = 0.f;
    if (p.m0 && slot >= 0 && on && row < p.A) {
      const int64_t at = p.transposed ? static_cast<int64_t>(col) * p.A + row
                                      : static_cast<int64_t>(row) * p.C + col;
      m[r] = p.m0[(slot * p.s.Hv + h) * head + at];
    }
  }
  float next = 0.f;  // backwards: the gate of the token after the current one
  const int n = t1 - t0;
  for (int base = 0; base < n; base += kTile) {
    const int count = min(kTile, n - base);
    __syncthreads();
    for (int e = threadIdx.x; e < count * p.A; e += kWarps * 32) {
      const int i = e / p.A, r = e % p.A;
      const int64_t t = REVERSE ? t1 - 1 - (base + i) : t0 + base + i;
      sa[i][r] = bf16_to_f32(p.a.p[t * p.a.st + ha * p.a.sh + r]);
      sb[i][r] = bf16_to_f32(p.b.p[t * p.b.st + hb * p.b.sh + r]);
    }
    if (threadIdx.x < count) {
      const int64_t t = REVERSE ? t1 - 1 - (base + threadIdx.x) : t0 + base + threadIdx.x;
      if (REVERSE)
        decay[threadIdx.x] = t + 1 < t1 ? expf(p.g.at(t + 1, h)) : 0.f;
      else
        decay[threadIdx.x] = expf(p.g.at(t, h));
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) {
      const int64_t t = REVERSE ? t1 - 1 - (base + i) : t0 + base + i;
      const float c = on ? bf16_to_f32(p.c.p[t * p.c.st + hc * p.c.sh + col]) : 0.f;
      const float d = decay[i];
      float acc = 0.f, ab = 0.f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        if (warp * ROWS + r < p.A) {
          const float av = sa[i][warp * ROWS + r], bv = sb[i][warp * ROWS + r];
          m[r] *= d;
          acc = fmaf(av, m[r], acc);
          ab = fmaf(av, bv, ab);
          m[r] = fmaf(bv, c, m[r]);
        }
      }
      part[i][warp][lane] = acc;
      if (lane == 0) own[i][warp] = ab;
    }
    __syncthreads();
    for (int i = warp; i < count; i += kWarps) {
      const int64_t t = REVERSE ? t1 - 1 - (base + i) : t0 + base + i;
      float y = 0.f, ab = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        y += part[i][w][lane];
        ab += own[i][w];
      }
      if (p.dots) {
        float dot = on ? y * bf16_to_f32(p.x.p[t * p.x.st + hc * p.x.sh + col]) : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0)
          p.dots[(static_cast<int64_t>(slice) * p.s.total + t) * p.s.Hv + h] = p.scale * dot;
      }
      if (on) y = fmaf(ab, bf16_to_f32(p.c.p[t * p.c.st + hc * p.c.sh + col]), y);
      y *= p.scale;
      if (on) {
        const int64_t at = (t * p.s.Hv + h) * p.C + col;
        if (p.out)
          p.out[at] = cconv::f32_to_bf16(y);
        else
          p.out32[at] = y;
      }
    }
  }
  if (!p.m1 || (p.status && p.status[0] != CCONV_OK)) return;
  if (REVERSE) next = n > 0 ? expf(p.g.at(t0, h)) : 0.f;
  const int64_t to = p.m1_slots ? slot : seq;
  if (to < 0) return;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int row = warp * ROWS + r;
    if (on && row < p.A) {
      const int64_t at = p.transposed ? static_cast<int64_t>(col) * p.A + row
                                      : static_cast<int64_t>(row) * p.C + col;
      p.m1[(to * p.s.Hv + h) * head + at] = (REVERSE ? next * p.m1_scale : p.m1_scale) * m[r];
    }
  }
}

// Sums the value heads of each query / key head: dst[t, hk, :] = sum over h of src[t, h, :].
// One warp for each (t, hk).
__global__ void __launch_bounds__(256)
    cattn_linear_heads_kernel(const float* src, LinearShape s, uint16_t* dst) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (w >= static_cast<int64_t>(s.total) * s.Hk) return;
  const int64_t t = w / s.Hk;
  const int hk = static_cast<int>(w % s.Hk), r = s.Hv / s.Hk;
  for (int c = lane; c < s.K; c += 32) {
    float sum = 0.f;
    for (int i = 0; i < r; ++i) sum += src[(t * s.Hv + static_cast<int64_t>(hk) * r + i) * s.K + c];
    dst[(t * s.Hk + hk) * s.K + c] = cconv::f32_to_bf16(sum);
  }
}

// dg_t = sum over i >= t of its sequence of (qdot_i - kdot_i).  One warp for each sequence and
// value head, walking from the last token in steps of 32.
__global__ void __launch_bounds__(128)
    cattn_linear_dg_kernel(const float* qdot, const float* kdot, int slices, LinearShape s,
                           const int32_t* cu, float* dg) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int lane = threadIdx.x % 32;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (w >= static_cast<int64_t>(s.nseq) * s.Hv) return;
  const int seq = static_cast<int>(w / s.Hv), h = static_cast<int>(w % s.Hv);
  int t0, t1;
  sequence_rows(cu, seq, s.total, t0, t1);
  const int64_t pitch = static_cast<int64_t>(s.total) * s.Hv;
  float carry = 0.f;
  for (int hi = t1; hi > t0; hi -= 32) {
    const int t = hi - 1 - lane;
    const int64_t at = static_cast<int64_t>(t) * s.Hv + h;
    float x = 0.f;
    if (t >= t0)
      for (int i = 0; i < slices; ++i) x += qdot[i * pitch + at] - kdot[i * pitch + at];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    x += carry;
    if (t >= t0) dg[at] = x;
    carry = __shfl_sync(0xffffffffu, x, 31);
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

static int check_states(const int32_t* cu, int64_t nseq, const float* initial, const float* fin,
                        const int32_t* idx, int64_t S, int32_t* status) {
  if (!cu) return CCONV_ERR_NULL;
  if (nseq < 1 || nseq > kMaxSeqs) return CCONV_ERR_SHAPE;
  if (!aligned(cu, 4)) return CCONV_ERR_ALIGN;
  if (idx) {
    if (!status) return CCONV_ERR_NULL;
    if (S < 1 || S > CCONV_UPDATE_MAX_SLOTS) return CCONV_ERR_SHAPE;
    if (!aligned(idx, 4) || !aligned(status, 4)) return CCONV_ERR_ALIGN;
  } else if ((initial || fin) && S < nseq) {
    return CCONV_ERR_SHAPE;
  }
  return aligned(initial, 16) && aligned(fin, 16) ? CCONV_OK : CCONV_ERR_ALIGN;
}

static int launch_sweep(const SweepArgs& p, bool reverse, cudaStream_t stream) {
  const int64_t slices = (p.C + kCols - 1) / kCols;
  const int64_t ctas = slices * p.s.Hv * p.s.nseq;
  if (ctas > (int64_t(1) << 31) - 1) return CCONV_ERR_SHAPE;
  const dim3 grid(static_cast<unsigned>(ctas)), block(kWarps * 32);
  cudaError_t e;
  if (p.A <= 128)
    e = reverse ? launch_pdl(cattn_linear_sweep_kernel<32, true>, grid, block, 0, stream, p)
                : launch_pdl(cattn_linear_sweep_kernel<32, false>, grid, block, 0, stream, p);
  else
    e = reverse ? launch_pdl(cattn_linear_sweep_kernel<64, true>, grid, block, 0, stream, p)
                : launch_pdl(cattn_linear_sweep_kernel<64, false>, grid, block, 0, stream, p);
  return e == cudaSuccess ? CCONV_OK : CCONV_ERR_CUDA;
}

static LinearShape shape_of(int64_t total, int64_t Hk, int64_t Hv, int64_t K, int64_t V,
                            int64_t nseq) {
  return LinearShape{static_cast<int>(total), static_cast<int>(Hk), static_cast<int>(Hv),
                     static_cast<int>(K), static_cast<int>(V), static_cast<int>(nseq)};
}

static Rows rows(const void* p, int64_t st, int64_t sh) {
  return Rows{static_cast<const uint16_t*>(p), st, sh};
}

static int64_t slices_of(int64_t C) { return (C + kCols - 1) / kCols; }

// Workspace of the backward: dq and dk of each value head, and their dots with q and k.
static size_t bwd_bytes(int64_t total, int64_t Hv, int64_t K) {
  return static_cast<size_t>(total) * Hv * (2 * K + 2 * slices_of(K)) * 4;
}

// CTAs of the chunked kernels: one per SM, or one per unit where there can be no more units.
static int chunk_grid(int64_t total, int64_t nseq, int64_t Hv, int64_t V, int* grid) {
  int dev = 0, sms = 0;
  if (report_cuda("cudaGetDevice", cudaGetDevice(&dev)) != cudaSuccess ||
      report_cuda("cudaDeviceGetAttribute",
                  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return CCONV_ERR_CUDA;
  const int64_t units = Hv * ((V + 127) / 128) * (total / 128 + nseq);
  *grid = static_cast<int>(units < sms ? units : sms);
  return CCONV_OK;
}

// The chunk offsets at the head of the workspace.
static size_t offsets_bytes(int64_t nseq) { return (static_cast<size_t>(nseq + 1) * 4 + 15) / 16 * 16; }

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
  if (rc == CCONV_OK) *bytes = bwd_bytes(total, Hv, K);
  return rc;
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
    rc = check_states(cu_seqlens, nseq, initial_state, final_state, state_indices, S, status_dev);
  if (rc != CCONV_OK) return rc;
  int grid = 0;
  if (chunk_grid(total, nseq, Hv, V, &grid) != CCONV_OK) return CCONV_ERR_CUDA;
  if (!workspace || workspace_bytes < offsets_bytes(nseq) + chunk_fwd_bytes(grid))
    return CCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
  int32_t* cstart = static_cast<int32_t*>(workspace);
  rc = launch_checks(state_indices, nseq, S, 0, status_dev, cu_seqlens, nseq, total, cstart, stream);
  if (rc != CCONV_OK) return rc;
  ChunkCall c{};
  c.q = rows(q, sqt, sqh), c.k = rows(k, skt, skh), c.v = rows(v, svt, svh);
  c.g = Gates{g, sgt, sgh};
  c.s = shape_of(total, Hk, Hv, K, V, nseq);
  c.cu = cu_seqlens, c.cstart = cstart;
  c.slots = Slots{state_indices, S};
  c.initial = initial_state, c.fin = final_state;
  c.status = state_indices ? status_dev : nullptr;
  c.scale = scale;
  c.o = static_cast<uint16_t*>(o);
  c.carry = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + offsets_bytes(nseq));
  c.grid = grid;
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
    rc = check_states(cu_seqlens, nseq, initial_state, nullptr, state_indices, S, status_dev);
  if (rc != CCONV_OK) return rc;
  if (!aligned(d_initial_state, 16)) return CCONV_ERR_ALIGN;
  if (total > 0) {
    if (!do_ || !dq || !dk || !dg) return CCONV_ERR_NULL;
    rc = check_rows(do_, total, Hv, sot, soh);
    if (rc != CCONV_OK) return rc;
    if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dg, 16)) return CCONV_ERR_ALIGN;
    if (!workspace || workspace_bytes < bwd_bytes(total, Hv, K)) return CCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
  }
  rc = launch_checks(state_indices, nseq, S, 0, status_dev, cu_seqlens, nseq, total, nullptr,
                     stream);
  if (rc != CCONV_OK) return rc;

  const Rows rq = rows(q, sqt, sqh), rk = rows(k, skt, skh), rv = rows(v, svt, svh),
             ro = rows(do_, sot, soh);
  float* part_q = static_cast<float*>(workspace);
  float* part_k = part_q + total * Hv * K;
  float* qdot = part_k + total * Hv * K;
  float* kdot = qdot + total * Hv * slices_of(K);
  SweepArgs base{};
  base.g = Gates{g, sgt, sgh};
  base.s = shape_of(total, Hk, Hv, K, V, nseq);
  base.cu = cu_seqlens;
  base.slots = Slots{state_indices, S};
  base.scale = scale;
  const int hk = base.s.Hk, hv = base.s.Hv;

  SweepArgs p = base;  // dq
  p.a = ro, p.ha = hv, p.b = rv, p.hb = hv, p.c = rk, p.hc = hk;
  p.A = base.s.V, p.C = base.s.K;
  p.m0 = initial_state, p.transposed = true;
  p.out32 = part_q, p.x = rq, p.dots = qdot;
  rc = launch_sweep(p, false, stream);
  if (rc != CCONV_OK) return rc;

  p = base;  // dk
  p.a = rv, p.ha = hv, p.b = ro, p.hb = hv, p.c = rq, p.hc = hk;
  p.A = base.s.V, p.C = base.s.K;
  p.out32 = part_k, p.x = rk, p.dots = kdot;
  rc = launch_sweep(p, true, stream);
  if (rc != CCONV_OK) return rc;

  p = base;  // dv, and the gradient of the initial states
  p.a = rk, p.ha = hk, p.b = rq, p.hb = hk, p.c = ro, p.hc = hv;
  p.A = base.s.K, p.C = base.s.V;
  p.out = static_cast<uint16_t*>(dv);
  p.m1 = d_initial_state, p.m1_scale = scale;
  rc = launch_sweep(p, true, stream);
  if (rc != CCONV_OK || total == 0) return rc;

  const unsigned warps = static_cast<unsigned>((total * Hk + 7) / 8);
  const unsigned lines = static_cast<unsigned>((nseq * Hv + 3) / 4);
  if (launch_pdl(cattn_linear_heads_kernel, dim3(warps), dim3(256), 0, stream,
                 static_cast<const float*>(part_q), base.s, static_cast<uint16_t*>(dq)) !=
          cudaSuccess ||
      launch_pdl(cattn_linear_heads_kernel, dim3(warps), dim3(256), 0, stream,
                 static_cast<const float*>(part_k), base.s, static_cast<uint16_t*>(dk)) !=
          cudaSuccess ||
      launch_pdl(cattn_linear_dg_kernel, dim3(lines), dim3(128), 0, stream,
                 static_cast<const float*>(qdot), static_cast<const float*>(kdot),
                 static_cast<int>(slices_of(K)), base.s, cu_seqlens, dg) != cudaSuccess)
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
