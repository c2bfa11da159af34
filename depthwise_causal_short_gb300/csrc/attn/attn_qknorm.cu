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
// sums over a head are a few shuffles; the rotation's partners exchange the raw bf16 words.  A
// group takes one token and kHeads of its heads at a time: the table row, fp32 and so twice the
// bytes of a head's channels, is read once for them, and all their loads are in flight
// together.  A CTA works on queries or on keys only, so that one set of weights (and of their
// sums) is live.  Four CTAs of 64 registers a thread forward and two of 128 backward: more (5 / 3)
// spill and take 1.2 times as long, and items of 2 or 8 heads, or the next item's channels fetched
// ahead, are slower as well.  16384 rows, 8 + 8 heads of 128: 25.3 us forward (5.5 TB/s of needed
// bytes), 41.7 us backward with the weights' gradients (4.9 TB/s).  Everything between the bf16 load and the one rounding at the store is fp32.
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
constexpr int kHeads = 4;  // heads of an item
constexpr int kFwdCtas = 4, kBwdCtas = 2;  // CTAs per SM of a full grid

struct Side {
  const uint16_t *x, *dy;
  uint16_t* out;  // y, or dx
  int64_t st, sh, dt, dh;
  const void* w;
  int H, heads, splits;  // heads; heads of an item (1 or kHeads); items of a token
  int64_t items;
};

struct NormArgs {
  Side side[2];  // queries, keys
  const float *cos, *sin;
  const int32_t* pos;
  float* part;  // backward: [grid][K] partial sums of the weights' gradients (NULL: not wanted)
  int64_t P;
  int ctas_q;   // CTAs of the queries; the others are the keys'
  int K, R, wdt;
  float inv;    // 1 / K or 1
  float eps;
};

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

__device__ __forceinline__ void load_weight(const void* w, int wdt, int c0, bool on, float* out) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    out[j] = !on ? 0.f
             : !w ? 1.f
             : wdt == CCONV_F32 ? static_cast<const float*>(w)[c0 + j]
                                : bf16_to_f32(static_cast<const uint16_t*>(w)[c0 + j]);
}

// The lane that holds the other channels of a lane's pairs: lanes [0, half) the first, lanes
// [half, 2 half) the second of each pair (itself for channels that are not rotated).
__device__ __forceinline__ int peer_of(int lane, int half) {
  return lane < half ? lane + half : lane < 2 * half ? lane - half : lane;
}

template <int LANES>
__device__ __forceinline__ uint4 exchange(const uint4& v, int peer) {
  return make_uint4(__shfl_sync(0xffffffffu, v.x, peer, LANES),
                    __shfl_sync(0xffffffffu, v.y, peer, LANES),
                    __shfl_sync(0xffffffffu, v.z, peer, LANES),
                    __shfl_sync(0xffffffffu, v.w, peer, LANES));
}

// A lane's 4 or 8 table entries in one access: as two, every line would be fetched twice.
__device__ __forceinline__ void ld_table(const float* p, float (&v)[8]) {
  asm volatile("ld.global.nc.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
                 "=f"(v[7])
               : "l"(p));
}
__device__ __forceinline__ void ld_table(const float* p, float (&v)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}

// The factors of a lane's 8 channels, in pairs: y = x . C + partner . S, where `partner` holds the
// other channel of each pair (partner_of).  Ones and zeros in the channels that are not rotated.
template <bool INTER>
__device__ __forceinline__ void load_angles(const NormArgs& p, int64_t at, int lane, float dir,
                                            f2* C, f2* S) {
#pragma unroll
  for (int j = 0; j < 4; ++j) C[j] = cconv::f2_splat(1.f), S[j] = 0;
  if (lane * 8 >= p.R) return;
  if (at < 0 || at >= p.P) {
    if (lane == 0) atomicOr(&g_fault_qknorm, kFaultPosition);
    at = at < 0 ? 0 : p.P - 1;
  }
  const int half = p.R / 2;
  const bool second = !INTER && lane * 8 >= half;
  const int64_t col = at * half + (INTER ? lane * 4 : second ? lane * 8 - half : lane * 8);
  if constexpr (INTER) {
    float c[4], s[4];
    ld_table(p.cos + col, c);
    ld_table(p.sin + col, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) C[j] = f2_pack(c[j], c[j]), S[j] = f2_pack(-dir * s[j], dir * s[j]);
  } else {
    float c[8], s[8];
    ld_table(p.cos + col, c);
    ld_table(p.sin + col, s);
    const f2 sign = cconv::f2_splat(second ? dir : -dir);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      C[j] = f2_pack(c[2 * j], c[2 * j + 1]);
      S[j] = cconv::f2_mul(sign, f2_pack(s[2 * j], s[2 * j + 1]));
    }
  }
}

// The words with the other channel of each pair: of the partner lane, or the own ones swapped.
template <int LANES, bool INTER>
__device__ __forceinline__ uint4 partner_of(const uint4& v, int peer) {
  if constexpr (INTER)
    return make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032),
                      __byte_perm(v.z, 0, 0x1032), __byte_perm(v.w, 0, 0x1032));
  return exchange<LANES>(v, peer);
}

__device__ __forceinline__ void unpack8(const uint4& v, f2* x) {
  x[0] = bf16x2_to_f2(v.x), x[1] = bf16x2_to_f2(v.y);
  x[2] = bf16x2_to_f2(v.z), x[3] = bf16x2_to_f2(v.w);
}
__device__ __forceinline__ uint4 pack8(const f2* x) {
  return make_uint4(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]), f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
}
template <int LANES>
__device__ __forceinline__ float group_dot(const f2* a, const f2* b) {
  f2 d = cconv::f2_mul(a[0], b[0]);
#pragma unroll
  for (int j = 1; j < 4; ++j) d = cconv::f2_fma(a[j], b[j], d);
  float d0, d1;
  f2_unpack(d, d0, d1);
  return group_sum<LANES>(d0 + d1);
}

// Where a group stands among its side's items (token, head block).
struct Cursor {
  int64_t it, step, items;
  int t, s, t_step, s_step, splits;
  __device__ __forceinline__ Cursor(const Side& side, int64_t first, int64_t stride)
      : it(first), step(stride), items(side.items), splits(side.splits) {
    t = static_cast<int>(it / splits), s = static_cast<int>(it % splits);
    t_step = static_cast<int>(step / splits), s_step = static_cast<int>(step % splits);
  }
  __device__ __forceinline__ void next() {  // without dividing
    it += step;
    t += t_step;
    s += s_step;
    if (s >= splits) s -= splits, ++t;
  }
};

// The table row of a cursor's token.  Read one item ahead, so that the table is fetched beside
// the channels and not one more latency behind them (16384 rows of 16 heads of 128: 27.9 to 25.3 us
// forward, 47.6 to 41.7 us backward).
__device__ __forceinline__ int64_t position(const NormArgs& p, const Cursor& at) {
  const int t = at.it < at.items ? at.t : 0;
  return p.pos && p.R > 0 ? __ldg(p.pos + t) : t;
}

template <int LANES, bool INTER>
__global__ void __launch_bounds__(kThreads, kFwdCtas)
    cattn_qknorm_fwd_kernel(const __grid_constant__ NormArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  constexpr int kGroups = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const bool on = lane * 8 < p.K;
  const bool isk = blockIdx.x >= p.ctas_q;
  const Side& side = p.side[isk];
  const int cta = isk ? blockIdx.x - p.ctas_q : blockIdx.x, ctas = isk ? gridDim.x - p.ctas_q : p.ctas_q;
  const int peer = INTER ? lane : peer_of(lane, p.R / 16);
  // The weights of each lane's channels and of the other ones of their pairs.
  __shared__ ulonglong2 weights[2][2][LANES];
  if (threadIdx.x < LANES) {
    float w[8], o[8];
    load_weight(side.w, p.wdt, lane * 8, on, w);
    load_weight(side.w, p.wdt, peer * 8, peer * 8 < p.K, o);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      weights[0][j][lane] = make_ulonglong2(f2_pack(w[4 * j], w[4 * j + 1]), f2_pack(w[4 * j + 2], w[4 * j + 3]));
      weights[1][j][lane] = INTER ? make_ulonglong2(f2_pack(o[4 * j + 1], o[4 * j]), f2_pack(o[4 * j + 3], o[4 * j + 2]))
                                  : make_ulonglong2(f2_pack(o[4 * j], o[4 * j + 1]), f2_pack(o[4 * j + 2], o[4 * j + 3]));
    }
  }
  __syncthreads();
  const int64_t st = side.st, sh = side.sh;
  const int H = side.H, heads = side.heads;
  // Whole warps walk the items together, so that every shuffle has its 32 lanes.
  const int64_t mine = (threadIdx.x % 32) / LANES;
  Cursor at(side, static_cast<int64_t>(cta) * kGroups + threadIdx.x / LANES,
            static_cast<int64_t>(ctas) * kGroups);
  int64_t row = position(p, at);
  while (at.it - mine < at.items) {
    const int64_t pos = row;
    const bool live = at.it < at.items;
    const int t = live ? at.t : 0, h0 = live ? at.s * heads : 0;
    const int n = live && on ? min(heads, H - h0) : 0;
    at.next();
    row = position(p, at);
    uint4 raw[kHeads];
    const uint16_t* x0 = side.x + t * st + h0 * sh + lane * 8;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, x0 += sh) {
      raw[i] = make_uint4(0, 0, 0, 0);
      if (i < n) raw[i] = ld_stream(x0);
    }
    // y = r (x . A + partner . B): weights and angles in one pair of factors a channel
    f2 A[4], B[4];
    load_angles<INTER>(p, pos, lane, 1.f, A, B);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const ulonglong2 w = weights[0][j][lane], o = weights[1][j][lane];
      A[2 * j] = cconv::f2_mul(A[2 * j], w.x), A[2 * j + 1] = cconv::f2_mul(A[2 * j + 1], w.y);
      B[2 * j] = cconv::f2_mul(B[2 * j], o.x), B[2 * j + 1] = cconv::f2_mul(B[2 * j + 1], o.y);
    }
    uint16_t* y0 = side.out + (static_cast<int64_t>(t) * H + h0) * p.K + lane * 8;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, y0 += p.K) {
      if (i >= heads) break;
      f2 x[4], o[4];
      unpack8(raw[i], x);
      const f2 r = cconv::f2_splat(rsqrtf(group_dot<LANES>(x, x) * p.inv + p.eps));
      unpack8(partner_of<LANES, INTER>(raw[i], peer), o);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = cconv::f2_mul(r, cconv::f2_fma(o[j], B[j], cconv::f2_mul(x[j], A[j])));
      if (i < n) *reinterpret_cast<uint4*>(y0) = pack8(x);
    }
  }
}

template <int LANES, bool INTER>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
    cattn_qknorm_bwd_kernel(const __grid_constant__ NormArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  constexpr int kGroups = kThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const bool on = lane * 8 < p.K;
  const bool isk = blockIdx.x >= p.ctas_q;
  const Side& side = p.side[isk];
  const int cta = isk ? blockIdx.x - p.ctas_q : blockIdx.x, ctas = isk ? gridDim.x - p.ctas_q : p.ctas_q;
  const int peer = INTER ? lane : peer_of(lane, p.R / 16);
  f2 w[4], dw[4];
  {
    float w1[8];
    load_weight(side.w, p.wdt, lane * 8, on, w1);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f2_pack(w1[2 * j], w1[2 * j + 1]), dw[j] = 0;
  }
  const int64_t st = side.st, sh = side.sh, dt = side.dt, dh = side.dh;
  const int H = side.H, heads = side.heads;
  const int64_t mine = (threadIdx.x % 32) / LANES;
  Cursor at(side, static_cast<int64_t>(cta) * kGroups + threadIdx.x / LANES,
            static_cast<int64_t>(ctas) * kGroups);
  int64_t row = position(p, at);
  while (at.it - mine < at.items) {
    const int64_t pos = row;
    const bool live = at.it < at.items;
    const int t = live ? at.t : 0, h0 = live ? at.s * heads : 0;
    const int n = live && on ? min(heads, H - h0) : 0;
    at.next();
    row = position(p, at);
    uint4 rx[kHeads], ry[kHeads];
    const uint16_t* x0 = side.x + t * st + h0 * sh + lane * 8;
    const uint16_t* d0 = side.dy + t * dt + h0 * dh + lane * 8;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, x0 += sh, d0 += dh) {
      rx[i] = ry[i] = make_uint4(0, 0, 0, 0);
      if (i < n) {
        rx[i] = ld_stream(x0);
        ry[i] = ld_stream(d0);
      }
    }
    f2 C[4], S[4];
    load_angles<INTER>(p, pos, lane, -1.f, C, S);
    uint16_t* y0 = side.out + (static_cast<int64_t>(t) * H + h0) * p.K + lane * 8;
#pragma unroll
    for (int i = 0; i < kHeads; ++i, y0 += p.K) {
      if (i >= heads) break;
      f2 x[4], d[4], o[4];
      unpack8(rx[i], x);
      unpack8(ry[i], d);
      unpack8(partner_of<LANES, INTER>(ry[i], peer), o);
      const float norm = group_dot<LANES>(x, x) * p.inv + p.eps;
      const f2 r = cconv::f2_splat(live && h0 + i < H ? rsqrtf(norm) : 0.f);  // no head: nothing to sum
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = cconv::f2_mul(x[j], r);
        d[j] = cconv::f2_fma(o[j], S[j], cconv::f2_mul(d[j], C[j]));
        dw[j] = cconv::f2_fma(d[j], x[j], dw[j]);
        d[j] = cconv::f2_mul(d[j], w[j]);
      }
      const f2 m = cconv::f2_splat(-group_dot<LANES>(d, x) * p.inv);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = cconv::f2_mul(r, cconv::f2_fma(x[j], m, d[j]));
      if (i < n) *reinterpret_cast<uint4*>(y0) = pack8(d);
    }
  }
  if (!p.part) return;
  // The CTA's sums: one row per group, added up group by group in a fixed order.
  __shared__ float rows[kGroups][LANES * 8 + 1];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f2_unpack(dw[j], rows[threadIdx.x / LANES][lane * 8 + 2 * j], rows[threadIdx.x / LANES][lane * 8 + 2 * j + 1]);
  __syncthreads();
  for (int c = threadIdx.x; c < p.K; c += kThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int gidx = 0; gidx < kGroups; ++gidx) s += rows[gidx][c];
    p.part[static_cast<int64_t>(blockIdx.x) * p.K + c] = s;
  }
}

// Adds the CTAs' partial sums in a fixed order: kReduceRows lanes of rows a column, then across
// them.  Columns of the queries' weights first, then the keys'.
constexpr int kReduceCols = 32, kReduceRows = 16;
__global__ void __launch_bounds__(kReduceCols* kReduceRows)
    cattn_qknorm_dw_kernel(const float* part, int ctas_q, int ctas, int K, int wdt, void* dwq, void* dwk) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float sums[kReduceRows][kReduceCols + 1];
  const int col = blockIdx.x * kReduceCols + threadIdx.x;
  const bool isk = col >= K;
  const int c = isk ? col - K : col;
  float s = 0.f;
  if (col < 2 * K) {
    const int first = isk ? ctas_q : 0, last = isk ? ctas : ctas_q;
#pragma unroll 8
    for (int i = first + threadIdx.y; i < last; i += kReduceRows) s += part[static_cast<int64_t>(i) * K + c];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || col >= 2 * K) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < kReduceRows; ++i) s += sums[i][threadIdx.x];
  void* dst = isk ? dwk : dwq;
  if (!dst) return;
  if (wdt == CCONV_F32)
    static_cast<float*>(dst)[c] = s;
  else
    static_cast<uint16_t*>(dst)[c] = cconv::f32_to_bf16(s);
}

static int lanes_of(int64_t K) { return K <= 32 ? 4 : K <= 64 ? 8 : K <= 128 ? 16 : 32; }

// Items and grid of a call: kHeads heads an item where that fills the machine, else one head;
// CTAs are dealt to queries and keys by their heads.
static int plan(NormArgs& p, int64_t total, int sms, int ctas_per_sm) {
  const int lanes = lanes_of(p.K), groups = kThreads / lanes;
  const int64_t all = p.side[0].H + p.side[1].H, most = static_cast<int64_t>(sms) * ctas_per_sm;
  const int heads = total * all >= most * groups * kHeads ? kHeads : 1;
  int64_t need[2];
  for (int i = 0; i < 2; ++i) {
    Side& s = p.side[i];
    s.heads = heads;
    s.splits = (s.H + heads - 1) / heads;
    s.items = total * s.splits;
    need[i] = (s.items + groups - 1) / groups;
  }
  int64_t q = need[0], k = need[1];
  if (q + k > most) {
    q = most * need[0] / (need[0] + need[1]);
    q = q < 1 ? 1 : q > most - 1 ? most - 1 : q;
    k = most - q;
  }
  p.ctas_q = static_cast<int>(q);
  return static_cast<int>(q + k);
}

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
    if (!aligned(p.cos, 32) || !aligned(p.sin, 32)) return CCONV_ERR_ALIGN;
    if (p.pos && !aligned(p.pos, 4)) return CCONV_ERR_ALIGN;
  }
  const size_t ew = wdt == CCONV_F32 ? 4 : 2;
  if (!aligned(p.side[0].w, ew) || !aligned(p.side[1].w, ew)) return CCONV_ERR_ALIGN;
  if (total == 0) return CCONV_OK;
  const Side &q = p.side[0], &k = p.side[1];
  if (!q.x || !k.x || !q.out || !k.out) return CCONV_ERR_NULL;
  int rc = check_rows(q.x, total, Hq, q.st, q.sh);
  if (rc == CCONV_OK) rc = check_rows(k.x, total, Hk, k.st, k.sh);
  if (rc != CCONV_OK) return rc;
  return aligned(q.out, 16) && aligned(k.out, 16) ? CCONV_OK : CCONV_ERR_ALIGN;
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
  p.side[0] = Side{static_cast<const uint16_t*>(q), nullptr, static_cast<uint16_t*>(yq), sqt, sqh, 0, 0,
                   wq, static_cast<int>(Hq), 0, 0, 0};
  p.side[1] = Side{static_cast<const uint16_t*>(k), nullptr, static_cast<uint16_t*>(yk), skt, skh, 0, 0,
                   wk, static_cast<int>(Hk), 0, 0, 0};
  p.cos = cos, p.sin = sin, p.pos = positions;
  const int rc = check(p, total, Hq, Hk, K, wdt, mode, eps, R, P);
  if (rc != CCONV_OK || total == 0) return rc;
  p.P = P, p.K = static_cast<int>(K), p.R = static_cast<int>(R), p.wdt = wdt;
  p.inv = mode == CATTN_NORM_RMS ? 1.f / static_cast<float>(K) : 1.f;
  p.eps = eps;
  int sms = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  const int grid = plan(p, total, sms, kFwdCtas);
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
  *bytes = static_cast<size_t>(sms) * kBwdCtas * static_cast<size_t>(K) * 4;
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
  p.side[0] = Side{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(dyq),
                   static_cast<uint16_t*>(dq), sqt, sqh, syqt, syqh, wq, static_cast<int>(Hq), 0, 0, 0};
  p.side[1] = Side{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(dyk),
                   static_cast<uint16_t*>(dk), skt, skh, sykt, sykh, wk, static_cast<int>(Hk), 0, 0, 0};
  p.cos = cos, p.sin = sin, p.pos = positions;
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
    if (!workspace || workspace_bytes < static_cast<size_t>(sms) * kBwdCtas * K * 4)
      return CCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
    p.part = static_cast<float*>(workspace);
  }
  p.P = P, p.K = static_cast<int>(K), p.R = static_cast<int>(R), p.wdt = wdt;
  p.inv = mode == CATTN_NORM_RMS ? 1.f / static_cast<float>(K) : 1.f;
  p.eps = eps;
  if (total > 0) {
    grid = plan(p, total, sms, kBwdCtas);
    if (launch_pdl(pick_bwd(lanes_of(K), interleaved != 0), dim3(grid), dim3(kThreads), 0, stream,
                   p) != cudaSuccess)
      return CCONV_ERR_CUDA;
  }
  if (!sums) return CCONV_OK;
  const int cols = static_cast<int>(2 * K);
  return launch_pdl(cattn_qknorm_dw_kernel, dim3((cols + kReduceCols - 1) / kReduceCols),
                    dim3(kReduceCols, kReduceRows), 0, stream,
                    static_cast<const float*>(workspace), p.ctas_q, grid, static_cast<int>(K),
                    static_cast<int>(wdt), dwq, dwk) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}
