// Host helpers shared by the library's translation units: error mapping, the
// device check, tensor maps and launch configurations.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "../../include/svdq.h"

namespace {

constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;  // 2 s per bounded wait

#define SVDQ_TRY(expr)                                              \
  do {                                                              \
    cudaError_t e_ = (expr);                                        \
    if (e_ != cudaSuccess) return e_ == cudaErrorMemoryAllocation   \
                               ? SVDQ_ERR_OOM : SVDQ_ERR_CUDA;      \
  } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

svdq_status check_device(int* dev_out, int* sms_out) {
  int dev = 0, n = 0;
  if (cudaGetDeviceCount(&n) != cudaSuccess || n == 0) {
    cudaGetLastError();
    return SVDQ_ERR_UNSUPPORTED_DEVICE;
  }
  if (cudaGetDevice(&dev) != cudaSuccess) return SVDQ_ERR_CUDA;
  int major = 0, minor = 0, sms = 0;
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  // the 4-bit tensor-core kernels are built for sm_100a only
  if (major != 10 || minor != 0) return SVDQ_ERR_UNSUPPORTED_DEVICE;
  if (dev_out) *dev_out = dev;
  if (sms_out) *sms_out = sms;
  return SVDQ_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 2-D tiled tensor map over a row-major [rows x cols] matrix (rows
// `row_bytes` apart; 0: packed).
svdq_status make_tmap(CUtensorMap* m, const void* ptr, CUtensorMapDataType dt, int elem_bytes,
                      uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows,
                      CUtensorMapSwizzle swz, uint64_t row_bytes = 0) {
  auto fn = encode_fn();
  if (!fn) return SVDQ_ERR_CUDA;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {row_bytes ? row_bytes : cols * static_cast<uint64_t>(elem_bytes)};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  CUresult r = fn(m, dt, 2, const_cast<void*>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SVDQ_OK : SVDQ_ERR_CUDA;
}

template <class K>
svdq_status set_smem(K kernel, int bytes) {
  SVDQ_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
  return SVDQ_OK;
}

// The dynamic shared-memory opt-in of kernel `Kern` on the current device.
// The attribute belongs to the device's context, so it is set once per
// device ordinal (bit `dev` of a per-kernel mask); two threads that race on a
// first call both set it, which is harmless.
template <auto Kern>
svdq_status ensure_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SVDQ_ERR_CUDA;
  const uint64_t bit = 1ull << dev;
  if (done.load(std::memory_order_acquire) & bit) return SVDQ_OK;
  svdq_status s = set_smem(Kern, bytes);
  if (s == SVDQ_OK) done.fetch_or(bit, std::memory_order_release);
  return s;
}

// Launch configuration with programmatic stream serialisation: the kernel may
// start (prologue: barrier set-up, tensor-memory allocation, tensor-map
// prefetch, weight loads) while the previous kernel of the stream finishes;
// every kernel of the library waits for that kernel (griddepcontrol.wait)
// before it reads or writes global memory the previous kernel may touch.
// `cluster` > 1 adds a cluster dimension.
struct LaunchCfg {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  LaunchCfg(dim3 grid, dim3 block, int smem, cudaStream_t st, int cluster = 1) {
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    int n = 1;
    if (cluster > 1) {
      attr[1].id = cudaLaunchAttributeClusterDimension;
      attr[1].val.clusterDim.x = cluster;
      attr[1].val.clusterDim.y = 1;
      attr[1].val.clusterDim.z = 1;
      n = 2;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
  }
};

}  // namespace
