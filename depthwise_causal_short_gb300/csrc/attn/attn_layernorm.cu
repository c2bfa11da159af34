// attn_layernorm.cu -- layer norm of rows or heads (or their norm by the root mean square), with weight,
// bias and the gate silu(z), and its gradient with the sums for weight and bias.
//
//   n = (x - m) r,  m = mean(x) (layer) or 0 (rms),  r = (mean((x - m)^2) + eps)^-1/2
//   y = (n w + b) silu(z)
//   du = dy silu(z),  dz = dy (n w + b) silu'(z),  dn = du w
//   dx = r (dn - n mean(dn n) - mean(dn)),  dw = sum of du n,  db = sum of du     (rms: no mean(dn))
//
// Bound by memory: every tensor is read or written once, and the gradient makes the statistics again
// from x, which it reads anyway: 16384 rows of 16 heads of 128 with a gate 31 us (6.5 TB/s, 96 % of a copy's rate),
// its gradient 55 (6.1, 90 %); 8192 rows of 4096 with a bias 23 and 44 (85 and 67 %: three sums across the
// CTA's warps a row, two CTAs of 128 registers a thread on an SM).  A group of GROUP threads owns a row, 8 channels (16 bytes) of each
// of PIECES pieces a thread; three rows ahead are on the way to shared memory.  The squares are
// summed after the mean is known (as sum(x^2) - C m^2 they would cancel for rows far from zero).
// The sums over rows stay in registers for all rows of a thread, meet in the CTA, and then, a row of
// the workspace for each CTA, in a second kernel; in the same order in every run.
#include "attn_chunk.cuh"

namespace cattn {

struct LnArgs {
  const uint16_t *x, *z, *dy;
  int64_t sxt, sxh, szt, szh, syt, syh;
  const void *w, *b;
  uint16_t *y, *dz;  // y, or dx
  float* part;       // [CTAs][2][C], or NULL
  int64_t rows;
  int H, C, wdt, layer;
  float count, inv, eps;  // C, 1 / C
};

constexpr int kLnThreads = 256;
constexpr int kLnAhead = 3;  // rows that the gradient's threads have on the way
constexpr int kMaxNorm = 8192;
constexpr int ln_threads(int group) { return group > kLnThreads ? group : group > 32 ? group : kLnThreads; }
// Threads an SM that a kernel's registers leave room for: the grids are that many, and each CTA goes on to
// the rows that are left.
// (16384 rows of 16 heads of 128: forward 31 us, 36 with room for 768, 34 for 1536; gradient 55, 59 with room for
// 768, 72 for 1024.)
constexpr int kLnFwdRoom = 1024, kLnBwdRoom = 512;

using cconv::f2_unpack;

// Eight values as four pairs.
__device__ __forceinline__ void widen(const uint4& raw, f2 (&x)[4]) {
  x[0] = bf16x2_to_f2(raw.x), x[1] = bf16x2_to_f2(raw.y), x[2] = bf16x2_to_f2(raw.z), x[3] = bf16x2_to_f2(raw.w);
}
__device__ __forceinline__ uint4 narrow(const f2 (&x)[4]) {
  return make_uint4(f2_to_bf16x2(x[0]), f2_to_bf16x2(x[1]), f2_to_bf16x2(x[2]), f2_to_bf16x2(x[3]));
}
__device__ __forceinline__ float both(f2 v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}
// Eight weights from channel c on.
__device__ __forceinline__ void load_weights(const void* w, int wdt, int c, float rest, bool on, f2 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_splat(rest);
  if (!w || !on) return;
  if (wdt == CCONV_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = f2_pack(__ldg(static_cast<const float*>(w) + c + 2 * i), __ldg(static_cast<const float*>(w) + c + 2 * i + 1));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned short* at = static_cast<const unsigned short*>(w) + c + 2 * i;
      x[i] = f2_pack(cconv::bf16_to_f32(__ldg(at)), cconv::bf16_to_f32(__ldg(at + 1)));
    }
  }
}
// 1 / (1 + e^-z)
__device__ __forceinline__ f2 sigmoid(f2 z) {
  float a, b;
  f2_unpack(f2_mul(z, f2_splat(-kLog2e)), a, b);
  return f2_pack(__fdividef(1.f, 1.f + exp2_fast(a)), __fdividef(1.f, 1.f + exp2_fast(b)));
}

// The sums of N values over the row's group, in every thread of it.  Across warps by shared memory, in turn
// through two buffers: whoever writes the one again has passed the barrier after the other's reads.  There
// the warps' values are read a lane each and added up by shuffles (all of them read by all threads, the
// sums were a third of the instructions for rows of 4096 channels).
template <int GROUP, int N>
__device__ __forceinline__ void group_sum(float (&a)[N], float2* buf, int& turn) {
#pragma unroll
  for (int o = (GROUP < 32 ? GROUP : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
  if constexpr (GROUP > 32) {
    constexpr int kGroupWarps = GROUP / 32;
    float2* at = buf + turn * 32;
    turn ^= 1;
    if (threadIdx.x % 32 == 0) at[threadIdx.x / 32] = make_float2(a[0], a[N - 1]);
    __syncthreads();
    const float2 v = at[threadIdx.x % kGroupWarps];
    a[0] = v.x, a[N - 1] = N > 1 ? v.y : v.x;
#pragma unroll
    for (int o = kGroupWarps / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
  }
}

// 16 bytes to shared memory, zeros (and nothing read) unless `in`.
__device__ __forceinline__ void copy_async(uint4* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(cconv::smem_addr(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

// Row (t, h) and the step to this group's next one.
struct RowWalk {
  int64_t r, step, t, dt;
  int h, dh, H;
  __device__ __forceinline__ RowWalk(int64_t first, int64_t by, int heads)
      : r(first), step(by), t(first / heads), dt(by / heads), h(static_cast<int>(first % heads)),
        dh(static_cast<int>(by % heads)), H(heads) {}
  __device__ __forceinline__ void next() {
    r += step;
    t += dt;
    h += dh;
    if (h >= H) h -= H, ++t;
  }
};

// Statistics of a row of x: x becomes n; returns r (0 for a row that is not there, whatever eps is).
template <int GROUP, int PIECES>
__device__ __forceinline__ float normalise(f2 (&x)[PIECES][4], const bool (&on)[PIECES], bool live, const LnArgs& p,
                                           float2* buf, int& turn) {
  if (p.layer) {
    f2 m = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = f2_add(m, x[i][j]);
    float mean[1] = {both(m)};
    group_sum<GROUP>(mean, buf, turn);
    // sum / C with one Newton step of the quotient: q = s inv is off by up to 2^-23 of itself (f), q + (s - q C) inv
    // by 2^-24 f and its rounding.  So a row of equal values, whose sum is exact, is its own mean; one step off,
    // the mean would be all that such a row's variance holds.  (8192 rows of 4096, gradient: 44.4 us; divided, 47.)
    const float q = mean[0] * p.inv;
    m = f2_splat(-fmaf(fmaf(-q, p.count, mean[0]), p.inv, q));
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = on[i] ? f2_add(x[i][j], m) : 0;
  }
  f2 q = 0;
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) q = f2_fma(x[i][j], x[i][j], q);
  float s[1] = {both(q)};
  group_sum<GROUP>(s, buf, turn);
  const float r = live ? rsqrtf(fmaf(s[0], p.inv, p.eps)) : 0.f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) x[i][j] = f2_mul(x[i][j], f2_splat(r));
  return r;
}

template <int GROUP, int PIECES, bool GATE>
__global__ void __launch_bounds__(ln_threads(GROUP)) cattn_layernorm_fwd_kernel(const LnArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float2 buf[64];
  int turn = 0;
  constexpr int kRows = ln_threads(GROUP) / GROUP;
  const int lane = threadIdx.x % GROUP;
  bool on[PIECES];
  f2 w[PIECES][4], b[PIECES][4];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int c = (lane + i * GROUP) * 8;
    on[i] = c < p.C;
    load_weights(p.w, p.wdt, c, 1.f, on[i], w[i]);
    load_weights(p.b, p.wdt, c, 0.f, on[i], b[i]);
  }
  RowWalk ahead(static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / GROUP,
                static_cast<int64_t>(gridDim.x) * kRows, p.H);
  int64_t next = ahead.r;
  // each thread copies its pieces of the rows ahead into a place of its own in shared memory
  extern __shared__ uint4 ring[];
  constexpr int kTensors = GATE ? 2 : 1, kThreads = ln_threads(GROUP);
  auto place = [&](int slot, int tensor, int i) { return ring + ((slot * kTensors + tensor) * PIECES + i) * kThreads + threadIdx.x; };
  int slot = 0;
  auto fetch = [&](int to) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (lane + i * GROUP) * 8;
      const bool in = ahead.r < p.rows && on[i];
      copy_async(place(to, 0, i), in ? p.x + ahead.t * p.sxt + ahead.h * p.sxh + c : p.x, in);
      if (GATE) copy_async(place(to, 1, i), in ? p.z + ahead.t * p.szt + ahead.h * p.szh + c : p.z, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead.next();
  };
#pragma unroll
  for (int i = 0; i < kLnAhead; ++i) fetch(i);
  // (whole warps, and with GROUP > 32 whole CTAs, leave the loop together)
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.rows;
       first += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = next;
    next += ahead.step;
    f2 x[PIECES][4];
    uint4 z[PIECES];
    asm volatile("cp.async.wait_group %0;" ::"n"(kLnAhead - 1) : "memory");
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      widen(*place(slot, 0, i), x[i]);
      if (GATE) z[i] = *place(slot, 1, i);
    }
    fetch(slot);
    slot = slot + 1 == kLnAhead ? 0 : slot + 1;
    normalise<GROUP, PIECES>(x, on, row < p.rows, p, buf, turn);
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if (!on[i]) continue;
        f2 g[4];
        if (GATE) widen(z[i], g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = f2_fma(x[i][j], w[i][j], b[i][j]);
          if (GATE) x[i][j] = f2_mul(x[i][j], f2_mul(g[j], sigmoid(g[j])));
        }
        __stcs(reinterpret_cast<uint4*>(p.y + row * p.C + (lane + i * GROUP) * 8), narrow(x[i]));
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// This CTA's sums s (of its groups' rows) to `dst` [C].
template <int GROUP, int PIECES>
__device__ __forceinline__ void put_sums(f2 (&s)[PIECES][4], const bool (&on)[PIECES], float* dst, int C,
                                         float* shared) {
  const int lane = threadIdx.x % GROUP;
  if constexpr (GROUP > 32) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if (on[i])
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<ulonglong2*>(dst + (lane + i * GROUP) * 8 + 4 * j) = make_ulonglong2(s[i][2 * j], s[i][2 * j + 1]);
  } else {
    constexpr int kWarps = kLnThreads / 32, kPitch = GROUP * PIECES * 8;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = 16; o >= GROUP; o >>= 1) s[i][j] = f2_add(s[i][j], __shfl_xor_sync(0xffffffffu, s[i][j], o));
        if (threadIdx.x % 32 < GROUP)
          *reinterpret_cast<f2*>(shared + threadIdx.x / 32 * kPitch + (lane + i * GROUP) * 8 + 2 * j) = s[i][j];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += kLnThreads) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) a += shared[i * kPitch + c];
      dst[c] = a;
    }
    __syncthreads();
  }
}

template <int GROUP, int PIECES, bool GATE>
__global__ void __launch_bounds__(ln_threads(GROUP), kLnBwdRoom / ln_threads(GROUP))
    cattn_layernorm_bwd_kernel(const LnArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float2 buf[64];
  __shared__ alignas(8) float shared[GROUP > 32 ? 1 : kLnThreads / 32 * GROUP * PIECES * 8];
  int turn = 0;
  constexpr int kRows = ln_threads(GROUP) / GROUP;
  const int lane = threadIdx.x % GROUP;
  bool on[PIECES];
  f2 w[PIECES][4], dw[PIECES][4], db[PIECES][4];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int c = (lane + i * GROUP) * 8;
    on[i] = c < p.C;
    load_weights(p.w, p.wdt, c, 1.f, on[i], w[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = 0;
  }
  RowWalk ahead(static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / GROUP,
                static_cast<int64_t>(gridDim.x) * kRows, p.H);
  int64_t next = ahead.r;
  // each thread copies its pieces of the rows ahead into a place of its own in shared memory
  extern __shared__ uint4 ring[];
  constexpr int kTensors = GATE ? 3 : 2, kThreads = ln_threads(GROUP);
  auto place = [&](int slot, int tensor, int i) { return ring + ((slot * kTensors + tensor) * PIECES + i) * kThreads + threadIdx.x; };
  int slot = 0;
  auto fetch = [&](int to) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int c = (lane + i * GROUP) * 8;
      const bool in = ahead.r < p.rows && on[i];
      copy_async(place(to, 0, i), in ? p.x + ahead.t * p.sxt + ahead.h * p.sxh + c : p.x, in);
      copy_async(place(to, 1, i), in ? p.dy + ahead.t * p.syt + ahead.h * p.syh + c : p.dy, in);
      if (GATE) copy_async(place(to, 2, i), in ? p.z + ahead.t * p.szt + ahead.h * p.szh + c : p.z, in);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ahead.next();
  };
#pragma unroll
  for (int i = 0; i < kLnAhead; ++i) fetch(i);
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.rows;
       first += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = next;
    next += ahead.step;
    f2 x[PIECES][4], du[PIECES][4];
    uint4 z[PIECES];
    asm volatile("cp.async.wait_group %0;" ::"n"(kLnAhead - 1) : "memory");
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      widen(*place(slot, 0, i), x[i]);
      widen(*place(slot, 1, i), du[i]);
      if (GATE) z[i] = *place(slot, 2, i);
    }
    fetch(slot);
    slot = slot + 1 == kLnAhead ? 0 : slot + 1;
    const float r = normalise<GROUP, PIECES>(x, on, row < p.rows, p, buf, turn);
    f2 dn_n = 0, dn = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      if (GATE) {
        f2 g[4], b[4];
        widen(z[i], g);
        load_weights(p.b, p.wdt, (lane + i * GROUP) * 8, 0.f, on[i], b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f2 one = f2_splat(1.f), minus = f2_splat(-1.f), s = sigmoid(g[j]), d = f2_mul(du[i][j], s);
          du[i][j] = f2_mul(d, g[j]);
          // silu'(z) = s (1 + z (1 - s))
          g[j] = f2_mul(f2_mul(d, f2_fma(x[i][j], w[i][j], b[j])), f2_fma(g[j], f2_fma(s, minus, one), one));
        }
        if (row < p.rows && on[i])
          __stcs(reinterpret_cast<uint4*>(p.dz + row * p.C + (lane + i * GROUP) * 8), narrow(g));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (rows and channels that are not there have du = 0; x is finite there)
        dw[i][j] = f2_fma(du[i][j], x[i][j], dw[i][j]);
        db[i][j] = f2_add(db[i][j], du[i][j]);
        du[i][j] = f2_mul(du[i][j], w[i][j]);
        dn_n = f2_fma(du[i][j], x[i][j], dn_n);
        dn = f2_add(dn, du[i][j]);
      }
    }
    float sums[2] = {both(dn_n), both(dn)};
    group_sum<GROUP>(sums, buf, turn);
    const f2 a = f2_splat(-sums[0] * p.inv), m = f2_splat(p.layer ? -sums[1] * p.inv : 0.f), scale = f2_splat(r);
    if (row < p.rows) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if (!on[i]) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = f2_mul(scale, f2_add(f2_fma(a, x[i][j], du[i][j]), m));
        __stcs(reinterpret_cast<uint4*>(p.y + row * p.C + (lane + i * GROUP) * 8), narrow(x[i]));
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (!p.part) return;
  float* dst = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.C;
  put_sums<GROUP, PIECES>(dw, on, dst, p.C, shared);
  put_sums<GROUP, PIECES>(db, on, dst + p.C, p.C, shared);
}

// dw and db from the CTAs' sums, one after the other in each of kSumRows parts, then these.
constexpr int kSumCols = 32, kSumRows = 16;
__global__ void __launch_bounds__(kSumCols * kSumRows)
    cattn_layernorm_sums_kernel(const float* part, int ctas, int C, int wdt, void* dw, void* db) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  __shared__ float sums[kSumRows][kSumCols];
  const int c = blockIdx.x * kSumCols + threadIdx.x;  // of 2 C
  float a = 0.f;
  if (c < 2 * C) {
#pragma unroll 8
    for (int i = threadIdx.y; i < ctas; i += kSumRows) a += __ldcs(part + static_cast<int64_t>(i) * 2 * C + c);
  }
  sums[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * C) return;
#pragma unroll
  for (int i = 1; i < kSumRows; ++i) a += sums[i][threadIdx.x];
  void* dst = c < C ? dw : db;
  if (!dst) return;
  if (wdt == CCONV_F32)
    static_cast<float*>(dst)[c % C] = a;
  else
    static_cast<uint16_t*>(dst)[c % C] = cconv::f32_to_bf16(a);
}

struct LnKernel {
  void (*run[2])(LnArgs);  // without a gate, with one
  int threads, rows;       // of a CTA
  int piece_bytes;         // shared memory of a tensor's rows ahead
  int room;
};
template <int GROUP, int PIECES, bool BWD>
static LnKernel kernel_of() {
  constexpr int threads = ln_threads(GROUP);
  LnKernel k{{}, threads, threads / GROUP, kLnAhead * PIECES * threads * 16, 0};
  if constexpr (BWD) {
    k.run[0] = cattn_layernorm_bwd_kernel<GROUP, PIECES, false>, k.run[1] = cattn_layernorm_bwd_kernel<GROUP, PIECES, true>;
    k.room = kLnBwdRoom;
  } else {
    k.run[0] = cattn_layernorm_fwd_kernel<GROUP, PIECES, false>, k.run[1] = cattn_layernorm_fwd_kernel<GROUP, PIECES, true>;
    k.room = kLnFwdRoom;
  }
  return k;
}
// The smallest group that holds a row in one piece a thread, to 128 channels, and in two above; in four in a
// forward without a gate, to 1024 (more tensors or more threads a row, and they cost more than they save), where
// that makes a CTA for each SM, and to 256 channels eight.  Four pieces over two, a forward's time, by rows:
//   256 channels    600 1.25   2400 1.12   4864 1.00   7000 1.10   14000 1.04   28000 1.03   40000 0.96  131072 0.87
//   512             600 1.14   1200 1.14   2400 0.84   4864 0.66   7000 0.89   14000 0.96   28000 0.92
//   1024            600 1.14   1200 0.74   2400 0.75   4864 1.10   7000 1.16   14000 1.06   28000 0.94  40000 0.92
// Measured, us, 33.5 million elements; pieces 1 / 2 / 4:
//   rows of 256     forward 21.9 / 21.8 / 18.9    with a gate 35.0 / 33.6 / 41.7    its gradient 71.3 / 60.7 / 136
//   512             29.5 / 25.3 / 20.6            - / 35.5 / 43.5                   without a gate 52.9 / 34.3 / 72
//   1024            30.3 / 26.0 / 24.0            40.9 / 36.3 / 46.9                52.5 / 40.6 / 78
//   4096            - / 23.4 / 26.0               - / 37.0 / 39.9                   57 / 43.2 / 83
template <bool BWD>
static LnKernel pick(int64_t C, bool gate, int64_t rows, int sms) {
  if (!BWD && !gate && C > 128 && C <= 1024) {
    const LnKernel four = C <= 256 ? kernel_of<8, 4, BWD>() : C <= 512 ? kernel_of<16, 4, BWD>() : kernel_of<32, 4, BWD>();
    if (rows >= static_cast<int64_t>(sms) * four.rows * (C <= 256 ? 8 : 1)) return four;
  }
  if (C <= 32) return kernel_of<4, 1, BWD>();
  if (C <= 64) return kernel_of<8, 1, BWD>();
  if (C <= 128) return kernel_of<16, 1, BWD>();
  if (C <= 256) return kernel_of<16, 2, BWD>();
  if (C <= 512) return kernel_of<32, 2, BWD>();
  if (C <= 1024) return kernel_of<64, 2, BWD>();
  if (C <= 2048) return kernel_of<128, 2, BWD>();
  if (C <= 4096) return kernel_of<256, 2, BWD>();
  return kernel_of<512, 2, BWD>();
}
static int64_t ctas_of(int64_t rows, const LnKernel& kern, int sms) {
  const int64_t ctas = (rows + kern.rows - 1) / kern.rows, most = static_cast<int64_t>(sms) * (kern.room / kern.threads);
  return ctas < most ? ctas : most;
}

static int launch_rows(void (*kernel)(LnArgs), const LnKernel& kern, int64_t ctas, int tensors, const LnArgs& a,
                       cudaStream_t stream) {
  const int bytes = tensors * kern.piece_bytes;
  if (bytes > 32 * 1024 && cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), bytes) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kern.threads), bytes, stream, a) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

static int check(const void* x, int64_t sxt, int64_t sxh, const void* z, int64_t szt, int64_t szh, int64_t total,
                 int64_t H, int64_t C, const void* w, const void* b, cconv_dtype wdt, cattn_norm mode, float eps) {
  if (total < 0 || total > kMaxRows || H < 1 || H > 65535 || C < 1 || C > kMaxNorm) return CCONV_ERR_SHAPE;
  if ((mode != CATTN_NORM_RMS && mode != CATTN_NORM_LAYER) || !(eps >= 0.f)) return CCONV_ERR_SHAPE;
  if (wdt != CCONV_F32 && wdt != CCONV_BF16) return CCONV_ERR_DTYPE;
  if (C % 8 != 0) return CCONV_ERR_ALIGN;
  const size_t ew = wdt == CCONV_F32 ? 4 : 2;
  if (!aligned(w, ew) || !aligned(b, ew)) return CCONV_ERR_ALIGN;
  if (total == 0) return CCONV_OK;
  if (!x) return CCONV_ERR_NULL;
  int rc = check_rows(x, total, H, sxt, sxh);
  if (rc == CCONV_OK && z) rc = check_rows(z, total, H, szt, szh);
  return rc;
}

static LnArgs args_of(const void* x, int64_t sxt, int64_t sxh, const void* z, int64_t szt, int64_t szh,
                      int64_t total, int64_t H, int64_t C, const void* w, const void* b, cconv_dtype wdt,
                      cattn_norm mode, float eps) {
  LnArgs a{};
  a.x = static_cast<const uint16_t*>(x), a.z = static_cast<const uint16_t*>(z);
  a.sxt = sxt, a.sxh = sxh, a.szt = szt, a.szh = szh;
  a.w = w, a.b = b;
  a.rows = total * H;
  a.H = static_cast<int>(H), a.C = static_cast<int>(C), a.wdt = wdt, a.layer = mode == CATTN_NORM_LAYER;
  a.count = static_cast<float>(C), a.inv = 1.f / a.count, a.eps = eps;
  return a;
}

}  // namespace cattn

extern "C" CCONV_API int cattn_layernorm_fwd(const void* x, int64_t sxt, int64_t sxh, const void* gate,
                                             int64_t szt, int64_t szh, int64_t total, int64_t H, int64_t C,
                                             const void* w, const void* b, cconv_dtype wdt, cattn_norm mode,
                                             float eps, void* y, cconv_stream_t stream) {
  using namespace cattn;
  const int rc = check(x, sxt, sxh, gate, szt, szh, total, H, C, w, b, wdt, mode, eps);
  if (rc != CCONV_OK || total == 0) return rc;
  if (!y) return CCONV_ERR_NULL;
  if (!aligned(y, 16)) return CCONV_ERR_ALIGN;
  LnArgs a = args_of(x, sxt, sxh, gate, szt, szh, total, H, C, w, b, wdt, mode, eps);
  a.y = static_cast<uint16_t*>(y);
  int sms = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  const LnKernel kern = pick<false>(C, gate != nullptr, a.rows, sms);
  const int64_t ctas = ctas_of(a.rows, kern, sms);
  return launch_rows(kern.run[gate != nullptr], kern, ctas, gate ? 2 : 1, a, stream);
}

extern "C" CCONV_API int cattn_layernorm_bwd_workspace_bytes(int64_t total, int64_t H, int64_t C, size_t* bytes) {
  using namespace cattn;
  if (!bytes) return CCONV_ERR_NULL;
  if (total < 0 || total > kMaxRows || H < 1 || H > 65535 || C < 1 || C > kMaxNorm) return CCONV_ERR_SHAPE;
  int sms = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  const LnKernel kern = pick<true>(C, false, total * H, sms);
  const int64_t ctas = ctas_of(total * H, kern, sms);
  *bytes = static_cast<size_t>(ctas > 0 ? ctas : 1) * 2 * static_cast<size_t>(C) * 4;
  return CCONV_OK;
}

extern "C" CCONV_API int cattn_layernorm_bwd(const void* x, int64_t sxt, int64_t sxh, const void* dy,
                                             int64_t syt, int64_t syh, const void* gate, int64_t szt,
                                             int64_t szh, int64_t total, int64_t H, int64_t C, const void* w,
                                             const void* b, cconv_dtype wdt, cattn_norm mode, float eps,
                                             void* dx, void* dgate, void* dw, void* db, void* workspace,
                                             size_t workspace_bytes, cconv_stream_t stream) {
  using namespace cattn;
  int rc = check(x, sxt, sxh, gate, szt, szh, total, H, C, w, b, wdt, mode, eps);
  if (rc != CCONV_OK) return rc;
  if (total > 0) {
    if (!dy || !dx || (gate && !dgate)) return CCONV_ERR_NULL;
    rc = check_rows(dy, total, H, syt, syh);
    if (rc != CCONV_OK) return rc;
    if (!aligned(dx, 16) || !aligned(dgate, 16)) return CCONV_ERR_ALIGN;
  }
  const size_t ew = wdt == CCONV_F32 ? 4 : 2;
  if (!aligned(dw, ew) || !aligned(db, ew)) return CCONV_ERR_ALIGN;
  LnArgs a = args_of(x, sxt, sxh, gate, szt, szh, total, H, C, w, b, wdt, mode, eps);
  a.dy = static_cast<const uint16_t*>(dy), a.syt = syt, a.syh = syh;
  a.y = static_cast<uint16_t*>(dx), a.dz = static_cast<uint16_t*>(dgate);
  int sms = 0;
  if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
  const LnKernel kern = pick<true>(C, gate != nullptr, a.rows, sms);
  const int64_t ctas = ctas_of(a.rows, kern, sms);
  const bool sums = dw || db;
  if (sums) {
    if (!workspace || workspace_bytes < static_cast<size_t>(ctas > 0 ? ctas : 1) * 2 * C * 4)
      return CCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
    a.part = static_cast<float*>(workspace);
  }
  if (total > 0 && launch_rows(kern.run[gate != nullptr], kern, ctas, gate ? 3 : 2, a, stream) != CCONV_OK)
    return CCONV_ERR_CUDA;
  if (!sums) return CCONV_OK;
  return launch_pdl(cattn_layernorm_sums_kernel, dim3(static_cast<unsigned>((2 * C + kSumCols - 1) / kSumCols)),
                    dim3(kSumCols, kSumRows), 0, stream, static_cast<const float*>(workspace),
                    static_cast<int>(ctas), static_cast<int>(C), static_cast<int>(wdt), dw, db) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}
