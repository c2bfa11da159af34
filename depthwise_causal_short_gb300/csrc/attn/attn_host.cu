// attn_host.cu -- what the entry points of libcattn share: launch recording, the device fault
// words, the check of state indices and row offsets.
#include <cudaTypedefs.h>

#include <cxxabi.h>

#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include "attn.cuh"

namespace cconv {

// The launch helper of common.cuh reports and records through these; each library has its own.
cudaError_t report_cuda(const char* what, cudaError_t e) {
  static const bool debug = getenv("CCONV_DEBUG") != nullptr;
  if (e != cudaSuccess && debug)
    fprintf(stderr, "cattn: %s failed: %s (%d)\n", what, cudaGetErrorString(e), static_cast<int>(e));
  return e;
}

struct LaunchRecord {
  const void* func;
  dim3 grid, block;
  size_t smem;
};
static thread_local bool t_recording = false;
static thread_local std::vector<LaunchRecord> t_records;

bool recording_launches() { return t_recording; }
void record_launch(const void* func, dim3 grid, dim3 block, size_t smem) {
  t_records.push_back(LaunchRecord{func, grid, block, smem});
}

int set_max_dynamic_smem(const void* func, int bytes) {
  return report_cuda("cudaFuncSetAttribute",
                     cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          bytes)) == cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cconv

namespace cattn {

static std::vector<int (*)(unsigned*)>& fault_readers() {
  static std::vector<int (*)(unsigned*)> v;
  return v;
}
FaultReader::FaultReader(int (*read)(unsigned*)) { fault_readers().push_back(read); }

static __device__ unsigned g_fault_host;

static int read_fault(unsigned* out) {
  const unsigned zero = 0;
  if (report_cuda("fault word", cudaMemcpyFromSymbol(out, g_fault_host, sizeof(*out))) !=
          cudaSuccess ||
      (*out && report_cuda("fault word", cudaMemcpyToSymbol(g_fault_host, &zero, sizeof(zero))) !=
                   cudaSuccess))
    return CCONV_ERR_CUDA;
  return CCONV_OK;
}
static FaultReader reader(read_fault);

// cuTensorMapEncodeTiled needs a context current on the calling thread, and a thread that has made
// no runtime call that binds one (autograd's workers) has none: cudaSetDevice on the current device
// binds its primary context.  Checked once per thread and device.
int bind_context() {
  static PFN_cuCtxGetCurrent_v4000 get = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
  });
  thread_local int bound = -1;
  int dev = 0;
  if (report_cuda("cudaGetDevice", cudaGetDevice(&dev)) != cudaSuccess) return CCONV_ERR_CUDA;
  if (bound == dev) return CCONV_OK;
  CUcontext ctx = nullptr;
  if ((!get || get(&ctx) != CUDA_SUCCESS || !ctx) &&
      report_cuda("cudaSetDevice", cudaSetDevice(dev)) != cudaSuccess)
    return CCONV_ERR_CUDA;
  bound = dev;
  return CCONV_OK;
}

// SMs of the current device.
int sm_count(int* sms) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (report_cuda("cudaGetDevice", cudaGetDevice(&dev)) != cudaSuccess) return CCONV_ERR_CUDA;
  if (dev >= 0 && dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return CCONV_OK;
  if (report_cuda("cudaDeviceGetAttribute",
                  cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return CCONV_ERR_CUDA;
  if (dev >= 0 && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
  return CCONV_OK;
}

constexpr int kCheckThreads = 512;

struct CheckArgs {
  const int32_t* idx;
  const int32_t* cu;
  int32_t* status;
  int32_t* cstart;
  int64_t S;
  int n, nseq, total, pad;
};

// One bit per slot in shared memory: a second claim of a slot is a repeat.
__global__ void __launch_bounds__(kCheckThreads) cattn_check_kernel(CheckArgs p) {
  extern __shared__ unsigned seen[];
  cconv::grid_dependency_wait();
  cconv::grid_launch_dependents();
  const int tid = threadIdx.x;
  if (p.cu) {
    bool bad = false;
    for (int i = tid; i <= p.nseq; i += kCheckThreads) {
      const int c = p.cu[i];
      bad |= i == 0 ? c != 0 : c < p.cu[i - 1];
      bad |= i == p.nseq && c != p.total;
    }
    bad = __syncthreads_or(bad);
    if (bad && tid == 0) atomicOr(&g_fault_host, kFaultSeqlens);
    if (p.cstart) {
      // running sum of the chunk counts, kCheckThreads sequences at a time
      __shared__ int sums[kCheckThreads / 32];
      int carry = 0;
      for (int at = 0; at < p.nseq; at += kCheckThreads) {
        const int i = at + tid;
        const int len = i < p.nseq && !bad ? p.cu[i + 1] - p.cu[i] : 0;
        int x = i < p.nseq && !bad ? max(1, (len + 127) / 128) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (tid % 32 >= o) x += y;
        }
        if (tid % 32 == 31) sums[tid / 32] = x;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kCheckThreads / 32; ++w) {
          if (w < tid / 32) x += sums[w];
          all += sums[w];
        }
        if (i < p.nseq) p.cstart[i + 1] = carry + x;
        carry += all;
        __syncthreads();
      }
      if (tid == 0) p.cstart[0] = 0;
    }
  }
  if (!p.idx) return;
  for (int i = tid; i < static_cast<int>((p.S + 31) / 32); i += kCheckThreads) seen[i] = 0;
  __shared__ unsigned offences;
  if (tid == 0) offences = 0;
  __syncthreads();
  unsigned bad = 0;
  for (int i = tid; i < p.n; i += kCheckThreads) {
    const int s = p.idx[i];
    if (s < 0) {
      if (!(p.pad && s == -1)) bad |= CCONV_IDX_NEGATIVE;
    } else if (s >= p.S) {
      bad |= CCONV_IDX_OUT_OF_RANGE;
    } else {
      const unsigned bit = 1u << (s & 31);
      if (atomicOr(&seen[s >> 5], bit) & bit) bad |= CCONV_IDX_DUPLICATE;
    }
  }
  if (bad) atomicOr(&offences, bad);
  __syncthreads();
  if (tid == 0) {
    p.status[0] = offences ? CCONV_ERR_INDEX : CCONV_OK;
    p.status[1] = static_cast<int>(offences);
  }
}

int launch_checks(const int32_t* idx, int64_t n, int64_t S, int pad, int32_t* status,
                  const int32_t* cu, int64_t nseq, int64_t total, int32_t* cstart,
                  cudaStream_t stream) {
  CheckArgs a{idx, cu, status, cstart, S, static_cast<int>(n), static_cast<int>(nseq),
              static_cast<int>(total), pad};
  const size_t smem = idx ? static_cast<size_t>((S + 31) / 32) * 4 : 0;
  if (smem > 32 * 1024 &&
      cconv::set_max_dynamic_smem(reinterpret_cast<const void*>(cattn_check_kernel),
                                  static_cast<int>(smem)) != CCONV_OK)
    return CCONV_ERR_CUDA;
  return launch_pdl(cattn_check_kernel, dim3(1), dim3(kCheckThreads), smem, stream, a) ==
                 cudaSuccess
             ? CCONV_OK
             : CCONV_ERR_CUDA;
}

}  // namespace cattn

extern "C" {

CCONV_API int cattn_describe_begin(void) {
  cconv::t_records.clear();
  cconv::t_recording = true;
  return CCONV_OK;
}

CCONV_API int cattn_describe_end(cconv_kernel_desc* out, int max, int* count) {
  using namespace cconv;
  t_recording = false;
  if (!count || (max > 0 && !out)) return CCONV_ERR_NULL;
  *count = static_cast<int>(t_records.size());
  int rc = CCONV_OK;
  for (int i = 0; i < max && i < static_cast<int>(t_records.size()); ++i) {
    const LaunchRecord& r = t_records[i];
    cconv_kernel_desc& d = out[i];
    memset(&d, 0, sizeof(d));
    cudaFuncAttributes fa{};
    int per_sm = 0;
    const int threads = static_cast<int>(r.block.x * r.block.y * r.block.z);
    if (report_cuda("cudaFuncGetAttributes", cudaFuncGetAttributes(&fa, r.func)) != cudaSuccess ||
        report_cuda("occupancy", cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                                     &per_sm, r.func, threads, r.smem)) != cudaSuccess) {
      rc = CCONV_ERR_CUDA;
      continue;
    }
    const char* mangled = nullptr;
    if (cudaFuncGetName(&mangled, r.func) == cudaSuccess && mangled) {
      int st = 0;
      char* dem = abi::__cxa_demangle(mangled, nullptr, nullptr, &st);
      snprintf(d.name, sizeof(d.name), "%s", st == 0 && dem ? dem : mangled);
      free(dem);
    }
    d.registers = fa.numRegs;
    d.local_bytes = static_cast<int>(fa.localSizeBytes);
    d.static_shared_bytes = static_cast<int>(fa.sharedSizeBytes);
    d.dynamic_shared_bytes = static_cast<int>(r.smem);
    d.threads = threads;
    d.ctas_per_sm = per_sm;
    d.ctas = static_cast<int64_t>(r.grid.x) * r.grid.y * r.grid.z;
  }
  t_records.clear();
  return rc;
}

CCONV_API int cattn_device_fault(int32_t* fault) {
  if (!fault) return CCONV_ERR_NULL;
  if (cudaDeviceSynchronize() != cudaSuccess) return CCONV_ERR_CUDA;
  unsigned all = 0;
  for (auto read : cattn::fault_readers()) {
    unsigned f = 0;
    const int rc = read(&f);
    if (rc != CCONV_OK) return rc;
    all |= f;
  }
  *fault = static_cast<int32_t>(all);
  return CCONV_OK;
}

}  // extern "C"
