// attn_update.cu -- linear attention's recurrent form for single tokens, on a pooled state.
//
//   S = exp(g) S + k v^T,  o = scale q^T S      for each row and value head
//
// Bound by memory: the fp32 state (64 KB a head at K = V = 128) is read and written once for
// some 5 fp32 operations a value.  A CTA owns a slice of V columns of one row and head: a warp
// reads whole 16-byte column quads of its K rows, so every access is a full line; all of a
// thread's loads are issued before the first is used.  256 rows of 16 heads of 128 x 128: 82.3 us,
// 6.4 TB/s (94 % of a copy's rate).  The K rows are dealt out to the
// warps, and their parts of o meet in shared memory in a fixed order.
#include "attn_linear.cuh"

namespace cattn {

using cconv::bf16_to_f32;

struct UpdateArgs {
  Rows q, k, v;
  Gates g;
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

// QUADS: column quads (4 columns) of a slice; 32 / QUADS rows of the state per warp access.
template <int QUADS>
__global__ void __launch_bounds__(kWarps * 32) cattn_linear_update_kernel(UpdateArgs p) {
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  constexpr int kPerWarp = 32 / QUADS;             // state rows of one warp access
  constexpr int kStep = kPerWarp * kWarps;         // and of the CTA's
  constexpr int kLoads = (kMaxK + kStep - 1) / kStep;
  __shared__ float qs[kMaxK], ks[kMaxK];
  __shared__ float4 part[kWarps * kPerWarp][QUADS];
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
  if (tid < p.K) {
    qs[tid] = p.scale * bf16_to_f32(p.q.p[i * p.q.st + hk * p.q.sh + tid]);
    ks[tid] = bf16_to_f32(p.k.p[i * p.k.st + hk * p.k.sh + tid]);
  }
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (on) {
    const uint2 raw = *reinterpret_cast<const uint2*>(p.v.p + i * p.v.st + h * p.v.sh + col);
    cconv::f2_unpack(cconv::bf16x2_to_f2(raw.x), v[0], v[1]);
    cconv::f2_unpack(cconv::bf16x2_to_f2(raw.y), v[2], v[3]);
  }
  const float a = expf(p.g.at(i, h));
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    const int r = row0 + j * kStep;
    if (on && r < p.K) {
      const float kk = ks[r], qq = qs[r];
      s[j].x = fmaf(a, s[j].x, kk * v[0]);
      s[j].y = fmaf(a, s[j].y, kk * v[1]);
      s[j].z = fmaf(a, s[j].z, kk * v[2]);
      s[j].w = fmaf(a, s[j].w, kk * v[3]);
      __stcs(S + r * pitch, s[j]);
      o.x = fmaf(qq, s[j].x, o.x);
      o.y = fmaf(qq, s[j].y, o.y);
      o.z = fmaf(qq, s[j].z, o.z);
      o.w = fmaf(qq, s[j].w, o.w);
    }
  }
  part[row0][quad] = o;
  __syncthreads();
  if (tid < QUADS && on) {
    o = part[0][tid];
#pragma unroll 8
    for (int r = 1; r < kWarps * kPerWarp; ++r) {
      const float4 x = part[r][tid];
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    const uint2 raw = make_uint2(cconv::f2_to_bf16x2(cconv::f2_pack(o.x, o.y)),
                                 cconv::f2_to_bf16x2(cconv::f2_pack(o.z, o.w)));
    *reinterpret_cast<uint2*>(p.o + (static_cast<int64_t>(i) * p.Hv + h) * p.V + col) = raw;
  }
}

}  // namespace cattn

extern "C" CCONV_API int cattn_linear_update(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
    int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh, int64_t N, int64_t Hk,
    int64_t Hv, int64_t K, int64_t V, float scale, float* state, int64_t S,
    const int32_t* state_indices, int pad_rows, void* o, int32_t* status_dev,
    cconv_stream_t stream) {
  using namespace cattn;
  if (N < 1) return CCONV_ERR_SHAPE;
  const int rc = check_linear(q, sqt, sqh, k, skt, skh, v, svt, svh, g, sgt, sgh, N, Hk, Hv, K, V, o);
  if (rc != CCONV_OK) return rc;
  if (!state || !status_dev) return CCONV_ERR_NULL;
  if (S < 1 || (state_indices ? S > CCONV_UPDATE_MAX_SLOTS : S < N)) return CCONV_ERR_SHAPE;
  if (!aligned(state, 16) || !aligned(status_dev, 4) || !aligned(state_indices, 4))
    return CCONV_ERR_ALIGN;
  // Up to 32 indices are checked by every warp of the update itself, which has to read them
  // anyway: one launch (1 row of 16 heads: 3.8 us against 4.6 with a checking kernel before it).
  const bool checked = state_indices && N > 32;
  if (checked && launch_checks(state_indices, N, S, pad_rows, status_dev, nullptr, 0, 0, nullptr,
                               stream) != CCONV_OK)
    return CCONV_ERR_CUDA;
  UpdateArgs a{};
  a.q = Rows{static_cast<const uint16_t*>(q), sqt, sqh};
  a.k = Rows{static_cast<const uint16_t*>(k), skt, skh};
  a.v = Rows{static_cast<const uint16_t*>(v), svt, svh};
  a.g = Gates{g, sgt, sgh};
  a.state = state;
  a.o = static_cast<uint16_t*>(o);
  a.slots = Slots{state_indices, S};
  a.status = status_dev;
  a.checked = checked;
  a.pad = pad_rows;
  a.scale = scale;
  a.N = static_cast<int>(N), a.Hk = static_cast<int>(Hk), a.Hv = static_cast<int>(Hv);
  a.K = static_cast<int>(K), a.V = static_cast<int>(V);
  const int quads = static_cast<int>(V / 4) >= 32 ? 32 : static_cast<int>(V / 4) > 8 ? 16 : 8;
  a.slices = static_cast<int>((V / 4 + quads - 1) / quads);
  const int64_t ctas = N * Hv * a.slices;
  if (ctas > (int64_t(1) << 31) - 1) return CCONV_ERR_SHAPE;
  auto kern = quads == 32   ? cattn_linear_update_kernel<32>
              : quads == 16 ? cattn_linear_update_kernel<16>
                            : cattn_linear_update_kernel<8>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), 0, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}
