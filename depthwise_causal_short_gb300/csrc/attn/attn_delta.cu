// attn_delta.cu -- the gated delta rule over packed sequences: the entry points.
#include "attn_delta.cuh"

namespace cattn {

constexpr int64_t kInKernelChecks = 32;  // state indices that the chain's CTAs check themselves
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;

static size_t record_bytes(int64_t total, int64_t nseq, int64_t Hv) {
  return total > 0 ? static_cast<size_t>(delta_slots(total, nseq) * Hv) * kRecordBytes : 0;
}
static uint8_t* align256(void* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 255) & ~static_cast<uintptr_t>(255));
}
static bool grids_fit(int64_t total, int64_t nseq, int64_t Hv, int64_t V) {
  return nseq * Hv * ((V + kColumns - 1) / kColumns) <= kMaxGrid && delta_slots(total, nseq) * Hv <= kMaxGrid;
}
static Rows rows(const void* p, int64_t st, int64_t sh) {
  return Rows{static_cast<const uint16_t*>(p), st, sh};
}

// What a backward call keeps in its workspace, from a 256-byte boundary.
struct DeltaWork {
  size_t records, z, u, heads, ends, rest, odots, vdots, bdots, sums, shut, anchors, adots, du, danchors, bytes;
  bool room;  // for both chains at once
};
// Both chains run at once where the device has room for both, with one sequence: up to half of the SMs.  With several,
// whose CTAs mostly end at different times, up to 5/8.  The gradient's time at once over in turn, by CTAs of a chain
// (152 SMs; heads of 128 x 128 or 128 x 96):
//   one sequence of 4096 rows           32 0.62   64 0.78   76 0.78   80 1.09   96 1.09   128 1.09
//   2 sequences, 3000 + 1000            72 0.78   88 0.81   96 0.81  112 0.92   128 0.92  144 0.93
//   4 to 7 uneven sequences, 4000       63 0.72   80 0.81   84 0.73   96 0.88   128 0.95  144 1.00
//   2 to 4 even ones of 1024 to 2048    64 0.87   72 0.89   80 1.08   96 1.17   128 1.30
// So from 77 CTAs to 95 even sequences lose 8 to 17 % and uneven ones win 20 %; the lengths are not known here.
static bool at_once(int64_t ctas, int64_t nseq, int sms) { return 8 * ctas <= (nseq > 1 ? 5 : 4) * int64_t(sms); }
constexpr int64_t kBothRoom = 96;  // the workspace, which no device is asked for, has room for it up to here
static DeltaWork delta_work(int64_t total, int64_t nseq, int64_t Hv, int64_t V) {
  const size_t tiles = static_cast<size_t>(delta_tiles(V)), rows = static_cast<size_t>(total) * Hv;
  const size_t states = total > 0 ? static_cast<size_t>(delta_slots(total, nseq)) * Hv * tiles * kStatePanel : 0;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += (n + 255) / 256 * 256;
    return r;
  };
  DeltaWork w{};
  w.records = take(record_bytes(total, nseq, Hv));
  w.z = take(states / kStatePanel * kDelta * kColumns * 4);
  w.u = take(states / kStatePanel * kUTile);
  w.heads = take(2 * states);
  w.ends = take(2 * states);
  w.rest = take(states / kStatePanel * kTokenPanel);
  w.odots = take(2 * tiles * rows * 4);
  w.vdots = take(2 * tiles * rows * 4);
  w.bdots = take(2 * tiles * rows * 4);
  w.sums = take(static_cast<size_t>(delta_slots(total, nseq)) * Hv * 8);
  w.shut = take(static_cast<size_t>(delta_slots(total, nseq)) * Hv * 4);
  const size_t anchors = total > 0 ? static_cast<size_t>(delta_anchors(total)) * Hv * tiles : 0;
  w.anchors = take(anchors * kAnchorFloats * 4);
  w.adots = take(anchors * kRowWarps * 4);
  w.room = total > 0 && nseq * Hv * static_cast<int64_t>(tiles) <= kBothRoom;
  if (w.room) {
    w.du = take(states / kStatePanel * kDelta * kColumns * 4);
    w.danchors = take(anchors * kAnchorFloats * 4);
  }
  w.bytes = at + 256;
  return w;
}

}  // namespace cattn

extern "C" CCONV_API int cattn_delta_fwd_workspace_bytes(int64_t total, int64_t nseq, int64_t Hk, int64_t Hv,
                                                         int64_t K, int64_t V, size_t* bytes) {
  using namespace cattn;
  if (!bytes) return CCONV_ERR_NULL;
  const int rc = check_sizes(total, nseq, Hk, Hv, K, V);
  if (rc != CCONV_OK) return rc;
  if (!grids_fit(total, nseq, Hv, V)) return CCONV_ERR_SHAPE;
  *bytes = record_bytes(total, nseq, Hv) + 256;
  return CCONV_OK;
}

extern "C" CCONV_API int cattn_delta_fwd(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
    int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh, const float* beta, int64_t sbt,
    int64_t sbh, int64_t total, int64_t Hk, int64_t Hv, int64_t K, int64_t V, const int32_t* cu_seqlens,
    int64_t nseq, float scale, const float* initial_state, float* final_state,
    const int32_t* state_indices, int64_t S, int32_t* status_dev, void* o, void* workspace,
    size_t workspace_bytes, cconv_stream_t stream) {
  using namespace cattn;
  int rc = check_linear(q, sqt, sqh, k, skt, skh, v, svt, svh, g, sgt, sgh, total, Hk, Hv, K, V, o);
  if (rc == CCONV_OK && total > 0) rc = check_gates(beta, total, Hv, sbt, sbh);
  if (rc == CCONV_OK)
    rc = check_states(cu_seqlens, nseq, Hv, initial_state, final_state, state_indices, S, status_dev);
  if (rc != CCONV_OK) return rc;
  if (!grids_fit(total, nseq, Hv, V)) return CCONV_ERR_SHAPE;
  if (!workspace || workspace_bytes < record_bytes(total, nseq, Hv) + 256) return CCONV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
  const bool checked = state_indices && nseq > kInKernelChecks;
  if (checked) {
    rc = launch_checks(state_indices, nseq, S, 0, status_dev, nullptr, 0, 0, nullptr, stream);
    if (rc != CCONV_OK) return rc;
  }
  DeltaCall c{};
  c.q = rows(q, sqt, sqh), c.k = rows(k, skt, skh), c.v = rows(v, svt, svh);
  c.g = Gates{g, sgt, sgh}, c.beta = Gates{beta, sbt, sbh};
  c.s = LinearShape{static_cast<int>(total), static_cast<int>(Hk), static_cast<int>(Hv),
                    static_cast<int>(K), static_cast<int>(V), static_cast<int>(nseq)};
  c.cu = cu_seqlens;
  c.slots = Slots{state_indices, S};
  c.checked = checked;
  c.status = status_dev;
  c.scale = scale;
  c.initial = initial_state, c.fin = final_state;
  c.o = static_cast<uint16_t*>(o);
  c.records = align256(workspace);
  if (total > 0) {
    rc = launch_delta_prep(c, stream);
    if (rc != CCONV_OK) return rc;
  }
  return launch_delta_fwd(c, stream);
}

extern "C" CCONV_API int cattn_delta_bwd_workspace_bytes(int64_t total, int64_t nseq, int64_t Hk, int64_t Hv,
                                                         int64_t K, int64_t V, size_t* bytes) {
  using namespace cattn;
  if (!bytes) return CCONV_ERR_NULL;
  const int rc = check_sizes(total, nseq, Hk, Hv, K, V);
  if (rc != CCONV_OK) return rc;
  if (!grids_fit(total, nseq, Hv, V)) return CCONV_ERR_SHAPE;
  *bytes = delta_work(total, nseq, Hv, V).bytes;
  return CCONV_OK;
}

extern "C" CCONV_API int cattn_delta_bwd(
    const void* q, int64_t sqt, int64_t sqh, const void* k, int64_t skt, int64_t skh, const void* v,
    int64_t svt, int64_t svh, const float* g, int64_t sgt, int64_t sgh, const float* beta, int64_t sbt,
    int64_t sbh, const void* do_, int64_t sot, int64_t soh, int64_t total, int64_t Hk, int64_t Hv, int64_t K,
    int64_t V, const int32_t* cu_seqlens, int64_t nseq, float scale, const float* initial_state,
    const int32_t* state_indices, int64_t S, int32_t* status_dev, void* dq, void* dk, void* dv, float* dg,
    float* dbeta, float* d_initial_state, void* workspace, size_t workspace_bytes, cconv_stream_t stream) {
  using namespace cattn;
  int rc = check_linear(q, sqt, sqh, k, skt, skh, v, svt, svh, g, sgt, sgh, total, Hk, Hv, K, V, dv);
  if (rc == CCONV_OK && total > 0) rc = check_gates(beta, total, Hv, sbt, sbh);
  if (rc == CCONV_OK)
    rc = check_states(cu_seqlens, nseq, Hv, initial_state, nullptr, state_indices, S, status_dev);
  if (rc != CCONV_OK) return rc;
  if (!aligned(d_initial_state, 32)) return CCONV_ERR_ALIGN;
  if (total > 0) {
    if (!do_ || !dq || !dk || !dg || !dbeta) return CCONV_ERR_NULL;
    rc = check_rows(do_, total, Hv, sot, soh);
    if (rc != CCONV_OK) return rc;
    if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dg, 16) || !aligned(dbeta, 16)) return CCONV_ERR_ALIGN;
  }
  if (!grids_fit(total, nseq, Hv, V)) return CCONV_ERR_SHAPE;
  const DeltaWork w = delta_work(total, nseq, Hv, V);
  if (total > 0) {
    if (!workspace || workspace_bytes < w.bytes) return CCONV_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return CCONV_ERR_ALIGN;
  }
  const bool checked = state_indices && (nseq > kInKernelChecks || total == 0);
  if (checked || total == 0) {
    rc = launch_checks(state_indices, nseq, S, 0, status_dev, total == 0 ? cu_seqlens : nullptr, nseq, total,
                       nullptr, stream);
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
  uint8_t* ws = align256(workspace);
  DeltaCall c{};
  c.q = rows(q, sqt, sqh), c.k = rows(k, skt, skh), c.v = rows(v, svt, svh), c.d_o = rows(do_, sot, soh);
  c.g = Gates{g, sgt, sgh}, c.beta = Gates{beta, sbt, sbh};
  c.s = LinearShape{static_cast<int>(total), static_cast<int>(Hk), static_cast<int>(Hv),
                    static_cast<int>(K), static_cast<int>(V), static_cast<int>(nseq)};
  c.cu = cu_seqlens;
  c.slots = Slots{state_indices, S};
  c.checked = checked;
  c.status = status_dev;
  c.scale = scale;
  c.initial = initial_state;
  c.records = ws + w.records;
  c.z = reinterpret_cast<float*>(ws + w.z);
  c.u = ws + w.u;
  c.heads = ws + w.heads, c.ends = ws + w.ends, c.rest = ws + w.rest;
  c.odots = reinterpret_cast<float*>(ws + w.odots);
  c.vdots = reinterpret_cast<float*>(ws + w.vdots);
  c.bdots = reinterpret_cast<float*>(ws + w.bdots);
  c.sums = reinterpret_cast<double*>(ws + w.sums);
  c.shut = reinterpret_cast<int*>(ws + w.shut);
  c.anchors = reinterpret_cast<float*>(ws + w.anchors);
  c.adots = reinterpret_cast<float*>(ws + w.adots);
  bool both = false;
  if (w.room) {
    int sms = 0;
    if (sm_count(&sms) != CCONV_OK) return CCONV_ERR_CUDA;
    both = at_once(nseq * Hv * delta_tiles(V), nseq, sms);
  }
  if (both) {
    c.du = reinterpret_cast<float*>(ws + w.du);
    c.danchors = reinterpret_cast<float*>(ws + w.danchors);
  }
  c.dq = static_cast<uint16_t*>(dq), c.dk = static_cast<uint16_t*>(dk), c.dv = static_cast<uint16_t*>(dv);
  c.dg = dg, c.dbeta = dbeta, c.dinit = d_initial_state;
  rc = launch_delta_prep(c, stream);
  if (both) {
    if (rc == CCONV_OK) rc = launch_delta_both(c, stream);
  } else {
    if (rc == CCONV_OK) rc = launch_delta_states(c, stream);
    if (rc == CCONV_OK) rc = launch_delta_back(c, stream);
  }
  if (rc == CCONV_OK) rc = launch_delta_grads(c, stream);
  if (rc == CCONV_OK) rc = launch_delta_gates(c, stream);
  return rc;
}
