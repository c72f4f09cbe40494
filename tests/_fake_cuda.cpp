// Stand-in for the CUDA runtime under the library's host code: two devices, no
// kernels.  It keeps the rules that the host code has to keep: a launch of more
// than 48 KB of dynamic shared memory fails unless the limit of that function
// was raised on the current device, and tensor maps are checked as the driver
// checks them; maps that reach beyond the one tensor that they begin in are
// counted (fake_tensor names the tensors).  Device memory is host memory that
// nothing writes.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <map>
#include <utility>

#define EXPORT extern "C" __attribute__((visibility("default")))

namespace {
int device = 0, launches = 0, last_device = -1, attribute_calls = 0, failing_attributes = 0, failing_launches = 0;
cudaError_t last_error = cudaSuccess;
std::map<std::pair<int, const void*>, int> limits;

std::map<uintptr_t, size_t> tensors;
int maps = 0, outside = 0;

bool within_one(uintptr_t from, uintptr_t to) {
  auto it = tensors.upper_bound(from);
  if (it == tensors.begin()) return false;
  --it;
  return to <= it->first + it->second;
}

cudaError_t answer(cudaError_t e) {
  if (e != cudaSuccess) last_error = e;
  return e;
}

CUresult encode(CUtensorMap*, CUtensorMapDataType dt, cuuint32_t rank, void* base, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t* steps, CUtensorMapInterleave,
                CUtensorMapSwizzle swizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  const uint64_t size = dt == CU_TENSOR_MAP_DATA_TYPE_UINT8 ? 1 : dt == CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 ? 2 : 4;
  bool ok = base && reinterpret_cast<uintptr_t>(base) % 16 == 0 && rank >= 1 && rank <= 5 && box[0] * size % 16 == 0;
  if (swizzle == CU_TENSOR_MAP_SWIZZLE_128B) ok = ok && box[0] * size <= 128;
  for (cuuint32_t i = 0; i < rank; ++i) ok = ok && dims[i] >= 1 && dims[i] <= 1ull << 32 && box[i] >= 1 &&
                                             box[i] <= 256 && steps[i] == 1;
  for (cuuint32_t i = 0; i + 1 < rank; ++i) ok = ok && strides[i] % 16 == 0 && strides[i] < 1ull << 40;
  uint64_t bytes = dims[0] * size;
  for (cuuint32_t i = 0; i + 1 < rank; ++i) bytes += (dims[i + 1] - 1) * strides[i];
  const uintptr_t at = reinterpret_cast<uintptr_t>(base);
  ++maps;
  outside += !within_one(at, at + bytes);
  return ok ? CUDA_SUCCESS : CUDA_ERROR_INVALID_VALUE;
}
}  // namespace

EXPORT void fake_set_device(int d) { device = d; }
EXPORT int fake_launches() { return launches; }
EXPORT int fake_last_device() { return last_device; }
EXPORT int fake_attribute_calls() { return attribute_calls; }
EXPORT void fake_tensor(void* p, size_t bytes) { tensors[reinterpret_cast<uintptr_t>(p)] = bytes; }
EXPORT void fake_forget_tensors() { tensors.clear(); }
EXPORT int fake_maps() { return maps; }
EXPORT int fake_maps_outside() { return outside; }
EXPORT void fake_fail_attributes(int n) { failing_attributes = n; }
EXPORT void fake_fail_launches(int n) { failing_launches = n; }

extern "C" {
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, CUstream_st*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) {
  ++launches;
  last_device = device;
  return cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  if (failing_launches > 0) {
    --failing_launches;
    return answer(cudaErrorLaunchOutOfResources);
  }
  const auto it = limits.find({device, f});
  if (c->dynamicSmemBytes > 48 * 1024 && (it == limits.end() || static_cast<int>(c->dynamicSmemBytes) > it->second))
    return answer(cudaErrorInvalidValue);
  if (!c->gridDim.x || c->gridDim.x > 0x7FFFFFFFu || c->gridDim.y > 65535 || !c->blockDim.x || c->blockDim.x > 1024)
    return answer(cudaErrorInvalidConfiguration);
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension && c->gridDim.x % c->attrs[i].val.clusterDim.x)
      return answer(cudaErrorInvalidConfiguration);
  ++launches;
  last_device = device;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int value) {
  ++attribute_calls;
  if (failing_attributes > 0) {
    --failing_attributes;
    return answer(cudaErrorMemoryAllocation);
  }
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) limits[{device, f}] = value;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
  if (limits.find({device, f}) == limits.end()) return answer(cudaErrorInvalidValue);
  *n = 0;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) {
      const unsigned x = c->attrs[i].val.clusterDim.x;      // as on a GB300, one CTA on an SM
      *n = x == 2 ? 76 : x == 4 ? 36 : x == 8 ? 15 : 0;
    }
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 0;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = std::aligned_alloc(256, (n + 255) / 256 * 256);
  if (*p) tensors[reinterpret_cast<uintptr_t>(*p)] = n;
  return *p ? cudaSuccess : answer(cudaErrorMemoryAllocation);
}
cudaError_t cudaFree(void* p) {
  tensors.erase(reinterpret_cast<uintptr_t>(p));
  std::free(p);
  return cudaSuccess;
}
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void* dst, const void*, size_t n, cudaMemcpyKind) {
  for (size_t i = 0; i < n; ++i) static_cast<char*>(dst)[i] = 0;
  return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}  // extern "C"
