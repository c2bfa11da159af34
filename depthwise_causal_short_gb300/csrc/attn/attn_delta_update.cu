// attn_delta_update.cu -- the gated delta rule's recurrent form for single tokens, on a pooled state.
//
//   z = v - a S^T k,  u = beta z,  S <- a S + k u^T,  o = scale S^T q     a = exp(g), for each row and head
//
// Bound by memory, as the linear attention's update: the fp32 state is read and written once.  A CTA
// owns a slice of V columns of one row and head and keeps it in registers; S^T k and S^T q are summed
// in one pass over it (o = scale (a S^T q + (q . k) u) needs no second one), the warps' parts meet in
// shared memory in a fixed order, and only then is the new state made and written.  So a CTA reads and writes
// by turns, and it takes several on an SM to keep memory busy: slices of 64 columns, three CTAs.  256 rows of
// 16 heads of 128 x 128: 84 us, 6.3 TB/s (94 % of a copy's rate); slices of 128 columns 118 us (two CTAs of 16
// warps 101), of 32 columns, half lines, 117.  (Heads of at most 32 columns: slices of 32, four CTAs an SM; 1024 rows
// of 16 heads 111 us, with half of a slice of 64 empty 123.)
#include "attn_linear.cuh"

namespace cattn {

using cconv::bf16_to_f32;

struct DeltaUpdateArgs {
  Rows q, k, v;
  Gates g, beta;
  float* state;
  uint16_t* o;
  Slots slots;
  int32_t* status;        // the verdict on state_indices
  int checked;            // it is there already; else each warp checks the (up to 32) indices
  int pad;
  float scale;
  int N, Hk, Hv, K, V;
  int slices;  // column slices of a head
};

constexpr int kWarps = 8;

__device__ __forceinline__ void add_scaled(float4& a, float w, const float4& x) {
  a.x = fmaf(w, x.x, a.x);
  a.y = fmaf(w, x.y, a.y);
  a.z = fmaf(w, x.z, a.z);
  a.w = fmaf(w, x.w, a.w);
}

// QUADS: column quads (4 columns) of a slice; 32 / QUADS rows of the state per warp access.  CTAS: on an SM.
template <int QUADS, int CTAS>
__global__ void __launch_bounds__(kWarps * 32, CTAS) cattn_delta_update_kernel(DeltaUpdateArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  constexpr int kPerWarp = 32 / QUADS;             // state rows of one warp access
  constexpr int kStep = kPerWarp * kWarps;         // and of the CTA's
  constexpr int kLoads = (kMaxK + kStep - 1) / kStep;
  __shared__ float qs[kMaxK], ks[kMaxK];
  __shared__ float4 part[2][kStep][QUADS];
  __shared__ float dots[kMaxK / 32];
  const int64_t cta = blockIdx.x;
  const int slice = static_cast<int>(cta % p.slices);
  const int h = static_cast<int>(cta / p.slices % p.Hv);
  const int i = static_cast<int>(cta / p.slices / p.Hv);
  const int tid = threadIdx.x;
  int64_t slot = i;
  if (p.checked) {
    if (p.status[0] != CCONV_OK) return;
    slot = p.slots.of(i);
  } else {
    unsigned bad = 0;
    if (p.slots.idx) {
      const int s = tid % 32 < p.N ? p.slots.idx[tid % 32] : -1;
      bad = check_indices(s, p.N, p.slots.S, p.pad, tid % 32);
      slot = __shfl_sync(0xffffffffu, s, i);
    }
    if (cta == 0 && tid == 0) {
      p.status[0] = bad ? CCONV_ERR_INDEX : CCONV_OK;
      p.status[1] = static_cast<int>(bad);
    }
    if (bad) return;
  }
  if (slot < 0) return;  // a padding row
  const int quad = tid % QUADS, row0 = tid / QUADS;
  const int col = (slice * QUADS + quad) * 4;
  const bool on = col < p.V;
  float4* S = reinterpret_cast<float4*>(p.state + ((slot * p.Hv + h) * p.K) * p.V + col);
  const int64_t pitch = p.V / 4;
  float4 s[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = row0 + j * kStep;
    if (on && r < p.K) s[j] = __ldcs(S + r * pitch);
  }
  const int hk = h / (p.Hv / p.Hk);
  if (tid < kMaxK) {
    float q = 0.f, k = 0.f;
    if (tid < p.K) {
      q = p.scale * bf16_to_f32(p.q.p[i * p.q.st + hk * p.q.sh + tid]);
      k = bf16_to_f32(p.k.p[i * p.k.st + hk * p.k.sh + tid]);
      qs[tid] = q;
      ks[tid] = k;
    }
    float d = q * k;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (tid % 32 == 0) dots[tid / 32] = d;
  }
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
    const uint2 raw = *reinterpret_cast<const uint2*>(p.v.p + i * p.v.st + h * p.v.sh + col);
    cconv::f2_unpack(cconv::bf16x2_to_f2(raw.x), v.x, v.y);
    cconv::f2_unpack(cconv::bf16x2_to_f2(raw.y), v.z, v.w);
  }
  const float a = expf(p.g.at(i, h)), beta = __ldg(p.beta.p + i * p.beta.st + h * p.beta.sh);
  __syncthreads();
  float4 sk = make_float4(0.f, 0.f, 0.f, 0.f), sq = sk;
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = row0 + j * kStep;
    if (on && r < p.K) {
      add_scaled(sk, ks[r], s[j]);
      add_scaled(sq, qs[r], s[j]);
    }
  }
  part[0][row0][quad] = sk;
  part[1][row0][quad] = sq;
  __syncthreads();
  if (!on) return;
  float4 u = part[0][0][quad];
#pragma unroll 8
  for (int r = 1; r < kStep; ++r) add_scaled(u, 1.f, part[0][r][quad]);
  u.x = beta * fmaf(-a, u.x, v.x);
  u.y = beta * fmaf(-a, u.y, v.y);
  u.z = beta * fmaf(-a, u.z, v.z);
  u.w = beta * fmaf(-a, u.w, v.w);
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = row0 + j * kStep;
    if (r < p.K) {
      const float kk = ks[r];
      s[j].x = fmaf(a, s[j].x, kk * u.x);
      s[j].y = fmaf(a, s[j].y, kk * u.y);
      s[j].z = fmaf(a, s[j].z, kk * u.z);
      s[j].w = fmaf(a, s[j].w, kk * u.w);
      __stcs(S + r * pitch, s[j]);
    }
  }
  if (tid < QUADS) {
    float4 o = part[1][0][tid];
#pragma unroll 8
    for (int r = 1; r < kStep; ++r) add_scaled(o, 1.f, part[1][r][tid]);
    const float d = (dots[0] + dots[1]) + (dots[2] + dots[3]);
    const uint2 raw = make_uint2(
        cconv::f2_to_bf16x2(cconv::f2_pack(fmaf(d, u.x, a * o.x), fmaf(d, u.y, a * o.y))),
        cconv::f2_to_bf16x2(cconv::f2_pack(fmaf(d, u.z, a * o.z), fmaf(d, u.w, a * o.w))));
    *reinterpret_cast<uint2*>(p.o + (static_cast<int64_t>(i) * p.Hv + h) * p.V + col) = raw;
  }
}

}  // namespace cattn

extern "C" CCONV_API int cattn_delta_update(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
    int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh, const float* beta, int64_t sbt,
    int64_t sbh, int64_t N, int64_t Hk, int64_t Hv, int64_t K, int64_t V, float scale, float* state,
    int64_t S, const int32_t* state_indices, int pad_rows, void* o, int32_t* status_dev,
    cconv_stream_t stream) {
  using namespace cattn;
  if (N < 1) return CCONV_ERR_SHAPE;
  int rc = check_linear(q, sqt, sqh, k, skt, skh, v, svt, svh, g, sgt, sgh, N, Hk, Hv, K, V, o);
  if (rc == CCONV_OK) rc = check_gates(beta, N, Hv, sbt, sbh);
  if (rc != CCONV_OK) return rc;
  if (!state || !status_dev) return CCONV_ERR_NULL;
  if (S < 1 || (state_indices ? S > CCONV_UPDATE_MAX_SLOTS : S < N)) return CCONV_ERR_SHAPE;
  if (!aligned(state, 16) || !aligned(status_dev, 4) || !aligned(state_indices, 4))
    return CCONV_ERR_ALIGN;
  const int quads = V > 32 ? 16 : 8;
  DeltaUpdateArgs a{};
  a.slices = static_cast<int>((V / 4 + quads - 1) / quads);
  const int64_t ctas = N * Hv * a.slices;
  if (ctas > (int64_t(1) << 31) - 1) return CCONV_ERR_SHAPE;
  // up to 32 indices are checked by every warp of the update itself: one launch
  const bool checked = state_indices && N > 32;
  if (checked && launch_checks(state_indices, N, S, pad_rows, status_dev, nullptr, 0, 0, nullptr,
                               stream) != CCONV_OK)
    return CCONV_ERR_CUDA;
  a.q = Rows{static_cast<const uint16_t*>(q), sqt, sqh};
  a.k = Rows{static_cast<const uint16_t*>(k), skt, skh};
  a.v = Rows{static_cast<const uint16_t*>(v), svt, svh};
  a.g = Gates{g, sgt, sgh};
  a.beta = Gates{beta, sbt, sbh};
  a.state = state;
  a.o = static_cast<uint16_t*>(o);
  a.slots = Slots{state_indices, S};
  a.status = status_dev;
  a.checked = checked;
  a.pad = pad_rows;
  a.scale = scale;
  a.N = static_cast<int>(N), a.Hk = static_cast<int>(Hk), a.Hv = static_cast<int>(Hv);
  a.K = static_cast<int>(K), a.V = static_cast<int>(V);
  auto kern = quads == 16 ? cattn_delta_update_kernel<16, 3> : cattn_delta_update_kernel<8, 4>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), 0, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}
