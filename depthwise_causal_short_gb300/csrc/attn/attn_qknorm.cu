// attn_qknorm.cu -- per-head norm of queries and keys with the position rotation in the same
// pass, and its gradient.
//
//   r = 1 / sqrt(m + eps), m = mean or sum of x^2 over the K channels of one head
//   u = w x r,  y = R(t) u;  R(t) turns pair p of the first R channels by the angle of row t
//   du = R(t)^T dy,  dn = w du,  n = x r
//   dx = r (dn - n * mean|sum(dn n)),  dw = sum over tokens and heads of du n
//
// Bound by memory: 4 bytes a channel forward, 6 backward, against some 10 fp32 operations.
// A group of 4 to 32 lanes holds one head (8 channels, one 16-byte access, a lane), so the
// sums over a head are a few shuffles.  A group takes one token and walks several of its heads:
// the table row is read once for them (it is fp32, twice the bytes of a head's channels), and
// kBatch heads' loads are in flight at once.  Everything between the bf16 load and the one
// rounding at the store is fp32.
#include "attn.cuh"

namespace cattn {

using cconv::bf16_to_f32;
using cconv::bf16x2_to_f2;
using cconv::f2;
using cconv::f2_pack;
using cconv::f2_to_bf16x2;
using cconv::f2_unpack;

static __device__ unsigned g_fault_qknorm;
static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_qknorm, sizeof(*out))) !=
          cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_qknorm, &zero,
                                                            sizeof(zero))) != cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

constexpr int kThreads = 256;
constexpr int kBatch = 4;      // heads in flight per group, forward
constexpr int kBatchBwd = 2;   // and backward (two tensors each)

struct NormArgs {
  const uint16_t *q, *k, *dyq, *dyk;
  uint16_t *oq, *ok;  // yq, yk or dq, dk
  int64_t sqt, sqh, skt, skh, syqt, syqh, sykt, sykh;
  const void *wq, *wk;
  const float *cos, *sin;
  const int32_t* pos;
  float* part;  // backward: [grid][2][K] partial sums of dwq, dwk (NULL: not wanted)
  int64_t P;
  int total, Hq, Hk, K, R, wdt;
  int heads;      // heads of one item
  int splits;     // items per token
  int64_t items;  // total * splits
  float inv;      // 1 / K or 1
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  f2_unpack(bf16x2_to_f2(v.x), x[0], x[1]);
  f2_unpack(bf16x2_to_f2(v.y), x[2], x[3]);
  f2_unpack(bf16x2_to_f2(v.z), x[4], x[5]);
  f2_unpack(bf16x2_to_f2(v.w), x[6], x[7]);
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(f2_to_bf16x2(f2_pack(x[0], x[1])), f2_to_bf16x2(f2_pack(x[2], x[3])),
                    f2_to_bf16x2(f2_pack(x[4], x[5])), f2_to_bf16x2(f2_pack(x[6], x[7])));
}
__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int LANES>
__device__ __forceinline__ float group_sum(float s) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o, LANES);
  return s;
}

// Turns the group's 8 channels a lane by `dir` * angle.  c, s: the lane's table entries (ones
// and zeros in the channels that are not rotated).
template <int LANES, bool INTER>
__device__ __forceinline__ void rotate(float* u, const float* c, const float* s, int lane, int half,
                                       float dir) {
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = u[2 * j], b = u[2 * j + 1], sn = dir * s[j];
      u[2 * j] = a * c[j] - b * sn;
      u[2 * j + 1] = b * c[j] + a * sn;
    }
  } else {
    // Lanes [0, half) hold the first channels of the pairs, lanes [half, 2 half) the second.
    const int peer = lane < half ? lane + half : lane < 2 * half ? lane - half : lane;
    const float sign = lane < half ? -dir : dir;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float other = __shfl_sync(0xffffffffu, u[j], peer, LANES);
      u[j] = u[j] * c[j] + other * (sign * s[j]);
    }
  }
}

__device__ __forceinline__ void load_weight(const void* w, int wdt, int c0, bool on, float* out) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    out[j] = !on ? 0.f
             : !w ? 1.f
             : wdt == CCONV_F32 ? static_cast<const float*>(w)[c0 + j]
                                : bf16_to_f32(static_cast<const uint16_t*>(w)[c0 + j]);
}

template <int LANES, bool INTER>
struct Angles {
  static constexpr int N = INTER ? 4 : 8;
  float c[N], s[N];
  __device__ __forceinline__ void load(const NormArgs& p, int t, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] = 1.f, s[j] = 0.f;
    if (lane * 8 >= p.R) return;
    int64_t at = p.pos ? p.pos[t] : t;
    if (at < 0 || at >= p.P) {
      if (lane == 0) atomicOr(&g_fault_qknorm, kFaultPosition);
      at = at < 0 ? 0 : p.P - 1;
    }
    const int half = p.R / 2;
    const int64_t col = INTER ? lane * 4 : (lane * 8 < half ? lane * 8 : lane * 8 - half);
    const float4* pc = reinterpret_cast<const float4*>(p.cos + at * half + col);
    const float4* ps = reinterpret_cast<const float4*>(p.sin + at * half + col);
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const float4 a = __ldg(pc + j), b = __ldg(ps + j);
      c[4 * j] = a.x, c[4 * j + 1] = a.y, c[4 * j + 2] = a.z, c[4 * j + 3] = a.w;
      s[4 * j] = b.x, s[4 * j + 1] = b.y, s[4 * j + 2] = b.z, s[4 * j + 3] = b.w;
    }
  }
};

template <int LANES, bool INTER>
__global__ void __launch_bounds__(kThreads) cattn_qknorm_fwd_kernel(NormArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  constexpr int kGroups = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const bool on = lane * 8 < p.K;
  float wq[8], wk[8];
  load_weight(p.wq, p.wdt, lane * 8, on, wq);
  load_weight(p.wk, p.wdt, lane * 8, on, wk);
  const int all = p.Hq + p.Hk;
  // Whole warps walk the items together, so that every shuffle has its 32 lanes.
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LANES;
  const int64_t warp0 = mine - (threadIdx.x % 32) / LANES;
  for (int64_t base = warp0, it = mine; base < p.items; base += step, it += step) {
    const bool live = it < p.items;
    const int t = live ? static_cast<int>(it / p.splits) : 0;
    const int h0 = live ? static_cast<int>(it % p.splits) * p.heads : 0;
    Angles<LANES, INTER> ang;
    ang.load(p, t, lane);
    for (int hb = 0; hb < p.heads; hb += kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + hb + i;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (live && on && hb + i < p.heads && h < all)
          raw[i] = ld_stream(h < p.Hq ? p.q + t * p.sqt + h * p.sqh + lane * 8
                                      : p.k + t * p.skt + (h - p.Hq) * p.skh + lane * 8);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int h = h0 + hb + i;
        const bool isq = h < p.Hq, used = live && hb + i < p.heads && h < all;
        float x[8];
        unpack8(raw[i], x);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        const float r = rsqrtf(group_sum<LANES>(ss) * p.inv + p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= r * (isq ? wq[j] : wk[j]);
        if (p.R > 0) rotate<LANES, INTER>(x, ang.c, ang.s, lane, p.R / 16, 1.f);
        if (used && on) {
          uint16_t* y = isq ? p.oq + (static_cast<int64_t>(t) * p.Hq + h) * p.K
                            : p.ok + (static_cast<int64_t>(t) * p.Hk + h - p.Hq) * p.K;
          *reinterpret_cast<uint4*>(y + lane * 8) = pack8(x);
        }
      }
    }
  }
}

template <int LANES, bool INTER>
__global__ void __launch_bounds__(kThreads) cattn_qknorm_bwd_kernel(NormArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  constexpr int kGroups = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const bool on = lane * 8 < p.K;
  float wq[8], wk[8], dwq[8], dwk[8];
  load_weight(p.wq, p.wdt, lane * 8, on, wq);
  load_weight(p.wk, p.wdt, lane * 8, on, wk);
#pragma unroll
  for (int j = 0; j < 8; ++j) dwq[j] = dwk[j] = 0.f;
  const int all = p.Hq + p.Hk;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kGroups + threadIdx.x / LANES;
  const int64_t warp0 = mine - (threadIdx.x % 32) / LANES;
  for (int64_t base = warp0, it = mine; base < p.items; base += step, it += step) {
    const bool live = it < p.items;
    const int t = live ? static_cast<int>(it / p.splits) : 0;
    const int h0 = live ? static_cast<int>(it % p.splits) * p.heads : 0;
    Angles<LANES, INTER> ang;
    ang.load(p, t, lane);
    for (int hb = 0; hb < p.heads; hb += kBatchBwd) {
      uint4 rx[kBatchBwd], ry[kBatchBwd];
#pragma unroll
      for (int i = 0; i < kBatchBwd; ++i) {
        const int h = h0 + hb + i;
        rx[i] = ry[i] = make_uint4(0, 0, 0, 0);
        if (live && on && hb + i < p.heads && h < all) {
          const bool isq = h < p.Hq;
          rx[i] = ld_stream(isq ? p.q + t * p.sqt + h * p.sqh + lane * 8
                                : p.k + t * p.skt + (h - p.Hq) * p.skh + lane * 8);
          ry[i] = ld_stream(isq ? p.dyq + t * p.syqt + h * p.syqh + lane * 8
                                : p.dyk + t * p.sykt + (h - p.Hq) * p.sykh + lane * 8);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatchBwd; ++i) {
        const int h = h0 + hb + i;
        const bool isq = h < p.Hq, used = live && hb + i < p.heads && h < all;
        float x[8], d[8];
        unpack8(rx[i], x);
        unpack8(ry[i], d);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
        const float norm = group_sum<LANES>(ss) * p.inv + p.eps;
        const float r = used ? rsqrtf(norm) : 0.f;  // no head: nothing for the weights' sums
        if (p.R > 0) rotate<LANES, INTER>(d, ang.c, ang.s, lane, p.R / 16, -1.f);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = x[j] * r, dn = d[j] * (isq ? wq[j] : wk[j]);
          if (isq)
            dwq[j] = fmaf(d[j], n, dwq[j]);
          else
            dwk[j] = fmaf(d[j], n, dwk[j]);
          dot = fmaf(dn, n, dot);
          x[j] = n;
          d[j] = dn;
        }
        const float m = group_sum<LANES>(dot) * p.inv;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = r * (d[j] - x[j] * m);
        if (used && on) {
          uint16_t* y = isq ? p.oq + (static_cast<int64_t>(t) * p.Hq + h) * p.K
                            : p.ok + (static_cast<int64_t>(t) * p.Hk + h - p.Hq) * p.K;
          *reinterpret_cast<uint4*>(y + lane * 8) = pack8(d);
        }
      }
    }
  }
  if (!p.part) return;
  // The CTA's sums: one row per group, added up group by group in a fixed order.
  __shared__ float rows[kGroups][LANES * 8 + 1];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int j = 0; j < 8; ++j) rows[threadIdx.x / LANES][lane * 8 + j] = side ? dwk[j] : dwq[j];
    __syncthreads();
    for (int c = threadIdx.x; c < p.K; c += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int gidx = 0; gidx < kGroups; ++gidx) s += rows[gidx][c];
      p.part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * p.K + c] = s;
    }
    __syncthreads();
  }
}

// Adds the CTAs' partial sums in a fixed order: 8 lanes of rows a column, then across them.
constexpr int kReduceCols = 32, kReduceRows = 16;
__global__ void __launch_bounds__(kReduceCols* kReduceRows)
    cattn_qknorm_dw_kernel(const float* part, int n, int K, int wdt, void* dwq, void* dwk) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float sums[kReduceRows][kReduceCols + 1];
  const int c = blockIdx.x * kReduceCols + threadIdx.x;
  float s = 0.f;
  if (c < 2 * K) {
#pragma unroll 8
    for (int i = threadIdx.y; i < n; i += kReduceRows) s += part[static_cast<int64_t>(i) * 2 * K + c];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * K) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kReduceRows; ++i) s += sums[i][threadIdx.x];
  void* dst = c < K ? dwq : dwk;
  if (!dst) return;
  const int at = c < K ? c : c - K;
  if (wdt == CCONV_F32)
    static_cast<float*>(dst)[at] = s;
  else
    static_cast<uint16_t*>(dst)[at] = cconv::f32_to_bf16(s);
}

static int sm_count(int* sms) {
  int dev = 0;
  if (report_cuda("cudaGetDevice", cudaGetDevice(&dev)) != cudaSuccess ||
      report_cuda("cudaDeviceGetAttribute",
                  cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}

static int lanes_of(int64_t K) { return K <= 32 ? 4 : K <= 64 ? 8 : K <= 128 ? 16 : 32; }

// Items and grid of a call.  With many tokens a group walks all heads of its token and the
// table row is read once; with few, heads are dealt out until the machine is full or each
// group has one batch.
static void plan(NormArgs& p, int sms, int batch, int ctas_per_sm, int* grid) {
  const int lanes = lanes_of(p.K), groups = kThreads / lanes;
  const int all = p.Hq + p.Hk;
  const int64_t full = static_cast<int64_t>(sms) * ctas_per_sm * groups;
  p.heads = (all + batch - 1) / batch * batch;
  while (p.heads > batch && static_cast<int64_t>(p.total) * ((all + p.heads - 1) / p.heads) < full)
    p.heads = (p.heads / 2 + batch - 1) / batch * batch;
  if (p.total < full / all) p.heads = 1;
  p.splits = (all + p.heads - 1) / p.heads;
  p.items = static_cast<int64_t>(p.total) * p.splits;
  const int64_t need = (p.items + groups - 1) / groups;
  const int64_t most = static_cast<int64_t>(sms) * ctas_per_sm;
  *grid = static_cast<int>(need < most ? need : most);
}

constexpr int kFwdCtas = 8, kBwdCtas = 4;  // CTAs per SM of a full grid

static int check(const NormArgs& p, int64_t total, int64_t Hq, int64_t Hk, int64_t K, int wdt,
                 int mode, float eps, int64_t R, int64_t P) {
  if (total < 0 || total > kMaxRows || Hq < 1 || Hk < 1 || Hq > 65535 || Hk > 65535 || K < 1 ||
      K > 256)
    return CCONV_ERR_SHAPE;
  if ((mode != CATTN_NORM_RMS && mode != CATTN_NORM_L2) || !(eps >= 0.f)) return CCONV_ERR_SHAPE;
  if (wdt != CCONV_BF16 && wdt != CCONV_F32) return CCONV_ERR_DTYPE;
  if (R < 0 || R > K) return CCONV_ERR_SHAPE;
  if (K % 8 != 0 || R % 16 != 0) return CCONV_ERR_ALIGN;
  if (R > 0) {
    if (!p.cos || !p.sin) return CCONV_ERR_NULL;
    if (P < 1 || (!p.pos && P < total)) return CCONV_ERR_SHAPE;
    if (!aligned(p.cos, 16) || !aligned(p.sin, 16)) return CCONV_ERR_ALIGN;
    if (p.pos && !aligned(p.pos, 4)) return CCONV_ERR_ALIGN;
  }
  const size_t ew = wdt == CCONV_F32 ? 4 : 2;
  if (!aligned(p.wq, ew) || !aligned(p.wk, ew)) return CCONV_ERR_ALIGN;
  if (total == 0) return CCONV_OK;
  if (!p.q || !p.k || !p.oq || !p.ok) return CCONV_ERR_NULL;
  int rc = check_rows(p.q, total, Hq, p.sqt, p.sqh);
  if (rc == CCONV_OK) rc = check_rows(p.k, total, Hk, p.skt, p.skh);
  if (rc != CCONV_OK) return rc;
  return aligned(p.oq, 16) && aligned(p.ok, 16) ? CCONV_OK : CCONV_ERR_ALIGN;
}

using Kernel = void (*)(NormArgs);
static Kernel pick_fwd(int lanes, bool inter) {
  switch (lanes) {
    case 4: return inter ? cattn_qknorm_fwd_kernel<4, true> : cattn_qknorm_fwd_kernel<4, false>;
    case 8: return inter ? cattn_qknorm_fwd_kernel<8, true> : cattn_qknorm_fwd_kernel<8, false>;
    case 16: return inter ? cattn_qknorm_fwd_kernel<16, true> : cattn_qknorm_fwd_kernel<16, false>;
    default: return inter ? cattn_qknorm_fwd_kernel<32, true> : cattn_qknorm_fwd_kernel<32, false>;
  }
}
static Kernel pick_bwd(int lanes, bool inter) {
  switch (lanes) {
    case 4: return inter ? cattn_qknorm_bwd_kernel<4, true> : cattn_qknorm_bwd_kernel<4, false>;
    case 8: return inter ? cattn_qknorm_bwd_kernel<8, true> : cattn_qknorm_bwd_kernel<8, false>;
    case 16: return inter ? cattn_qknorm_bwd_kernel<16, true> : cattn_qknorm_bwd_kernel<16, false>;
    default: return inter ? cattn_qknorm_bwd_kernel<32, true> : cattn_qknorm_bwd_kernel<32, false>;
  }
}

}  // namespace cattn

extern "C" CCONV_API int cattn_qknorm_fwd(const void* q, int64_t sqt, int64_t sqh, const void* k,
                                          int64_t skt, int64_t skh, int64_t total, int64_t Hq,
                                          int64_t Hk, int64_t K, const void* wq, const void* wk,
                                          cconv_dtype wdt, cattn_norm mode, float eps,
                                          const float* cos, const float* sin, int64_t P, int64_t R,
                                          int interleaved, const int32_t* positions, void* yq,
                                          void* yk, cconv_stream_t stream) {
  using namespace cattn;
  NormArgs p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.oq = static_cast<uint16_t*>(yq);
  p.ok = static_cast<uint16_t*>(yk);
  p.sqt = sqt, p.sqh = sqh, p.skt = skt, p.skh = skh;
  p.wq = wq, p.wk = wk, p.cos = cos, p.sin = sin, p.pos = positions;
  const int rc = check(p, total, Hq, Hk, K, wdt, mode, eps, R, P);
  if (rc != CCONV_OK || total == 0) return rc;
  p.P = P, p.total = static_cast<int>(total), p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk), p.K = static_cast<int>(K), p.R = static_cast<int>(R), p.wdt = wdt;
  p.inv = mode == CATTN_NORM_RMS ? 1.f / static_cast<float>(K) : 1.f;
  p.eps = eps;
  int sms = 0, grid = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  plan(p, sms, kBatch, kFwdCtas, &grid);
  return launch_pdl(pick_fwd(lanes_of(K), interleaved != 0), dim3(grid), dim3(kThreads), 0, stream,
                    p) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

extern "C" CCONV_API int cattn_qknorm_bwd_workspace_bytes(int64_t total, int64_t Hq, int64_t Hk,
                                                          int64_t K, size_t* bytes) {
  using namespace cattn;
  if (!bytes) return CCONV_ERR_NULL;
  if (total < 0 || total > kMaxRows || Hq < 1 || Hk < 1 || K < 1 || K > 256) return CCONV_ERR_SHAPE;
  int sms = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  *bytes = static_cast<size_t>(sms) * kBwdCtas * 2 * static_cast<size_t>(K) * 4;
  return CCONV_OK;
}

extern "C" CCONV_API int cattn_qknorm_bwd(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh,
    const void* dyq, int64_t syqt, int64_t syqh, const void* dyk, int64_t sykt, int64_t sykh,
    int64_t total, int64_t Hq, int64_t Hk, int64_t K, const void* wq, const void* wk,
    cconv_dtype wdt, cattn_norm mode, float eps, const float* cos, const float* sin, int64_t P,
    int64_t R, int interleaved, const int32_t* positions, void* dq, void* dk, void* dwq, void* dwk,
    void* workspace, size_t workspace_bytes, cconv_stream_t stream) {
  using namespace cattn;
  NormArgs p{};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.dyq = static_cast<const uint16_t*>(dyq);
  p.dyk = static_cast<const uint16_t*>(dyk);
  p.oq = static_cast<uint16_t*>(dq);
  p.ok = static_cast<uint16_t*>(dk);
  p.sqt = sqt, p.sqh = sqh, p.skt = skt, p.skh = skh;
  p.syqt = syqt, p.syqh = syqh, p.sykt = sykt, p.sykh = sykh;
  p.wq = wq, p.wk = wk, p.cos = cos, p.sin = sin, p.pos = positions;
  int rc = check(p, total, Hq, Hk, K, wdt, mode, eps, R, P);
  if (rc != CCONV_OK) return rc;
  if (total > 0) {
    if (!dyq || !dyk) return CCONV_ERR_NULL;
    rc = check_rows(dyq, total, Hq, syqt, syqh);
    if (rc == CCONV_OK) rc = check_rows(dyk, total, Hk, sykt, sykh);
    if (rc != CCONV_OK) return rc;
  }
  const size_t ew = wdt == CCONV_F32 ? 4 : 2;
  if (!aligned(dwq, ew) || !aligned(dwk, ew)) return CCONV_ERR_ALIGN;
  int sms = 0, grid = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  const bool sums = dwq || dwk;
  if (sums) {
    if (!workspace || workspace_bytes < static_cast<size_t>(sms) * kBwdCtas * 2 * K * 4)
      return CCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
    p.part = static_cast<float*>(workspace);
  }
  p.P = P, p.total = static_cast<int>(total), p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk), p.K = static_cast<int>(K), p.R = static_cast<int>(R), p.wdt = wdt;
  p.inv = mode == CATTN_NORM_RMS ? 1.f / static_cast<float>(K) : 1.f;
  p.eps = eps;
  if (total > 0) {
    plan(p, sms, kBatchBwd, kBwdCtas, &grid);
    if (launch_pdl(pick_bwd(lanes_of(K), interleaved != 0), dim3(grid), dim3(kThreads), 0, stream,
                   p) != cudaSuccess)
      return CCONV_ERR_CUDA;
  }
  if (!sums) return CCONV_OK;
  const int cols = static_cast<int>(2 * K);
  return launch_pdl(cattn_qknorm_dw_kernel, dim3((cols + kReduceCols - 1) / kReduceCols),
                    dim3(kReduceCols, kReduceRows), 0, stream,
                    static_cast<const float*>(workspace), grid, static_cast<int>(K),
                    static_cast<int>(wdt), dwq, dwk) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}
