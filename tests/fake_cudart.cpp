// A stand-in for the CUDA runtime: the host code of the cache operators links against
// it in place of the real one, so that its calls, its launches and what it makes of
// their errors can be tested without a device.  Nothing runs on one.
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include <cuda_runtime.h>

namespace {
std::mutex lock;
// (functions, since registration comes before this file's own constructors)
std::map<const void*, std::string>& kernels() {  // host stub -> kernel name
  static std::map<const void*, std::string> m;
  return m;
}
std::map<std::string, void*>& variables() {  // device variable -> its host shadow
  static std::map<std::string, void*> m;
  return m;
}
std::vector<std::string> launched;
std::string failing;  // the call that fails next, and after how many more of it
int failing_after, failing_with;
thread_local cudaError_t last = cudaSuccess;
int poke_value, poke_after;  // written to poke_name by the next synchronisation but so many
std::string poke_name;

cudaError_t result(const char* call) {
  std::lock_guard<std::mutex> g(lock);
  if (failing == call && failing_after-- == 0) {
    failing.clear();
    return last = (cudaError_t)failing_with;
  }
  return cudaSuccess;
}

int encoder(void*, ...) { return 0; }

int* variable(const std::string& name) {
  for (auto& v : variables())
    if (v.first.find(name) != std::string::npos) return (int*)v.second;
  return nullptr;
}
}  // namespace

extern "C" {
// ---- for the tests ----
void fake_reset() {
  std::lock_guard<std::mutex> g(lock);
  launched.clear();
  failing.clear();
  poke_name.clear();
  last = cudaSuccess;
  for (auto& v : variables()) memset(v.second, 0, sizeof(int));
}
void fake_fail(const char* call, int after, int error) {
  failing = call;
  failing_after = after;
  failing_with = error;
}
void fake_pending(int error) { last = (cudaError_t)error; }
int fake_peek() { return last; }
int fake_launches() { return (int)launched.size(); }
const char* fake_launch(int i) { return launched[i].c_str(); }
void fake_set(const char* name, int value) { *variable(name) = value; }
int fake_get(const char* name) { return *variable(name); }
void fake_poke_at_sync(const char* name, int value, int after) {
  poke_name = name;
  poke_after = after;
  poke_value = value;
}

// ---- the runtime ----
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* stub, char*, const char* name, int, uint3*, uint3*, dim3*,
                            dim3*, int*) {
  kernels()[stub] = name;
}
void __cudaRegisterVar(void**, char* shadow, char*, const char* name, int, size_t, int, int) {
  variables()[name] = shadow;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* stub) {
  *k = (cudaKernel_t)stub;
  return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void*) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) {
  return cudaErrorNotSupported;  // every launch goes through cudaLaunchKernelExC
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void* stub, void**) {
  const cudaError_t e = result("launch");
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> g(lock);
  launched.push_back(kernels()[stub]);
  if (launched.back().find("kv_status_take") != std::string::npos) {
    *variable("kv_status_taken") = *variable("kv_status_word");
    *variable("kv_status_word") = 0;
  }
  return cudaSuccess;
}
cudaError_t cudaMemcpyFromSymbolAsync(void* to, const void* symbol, size_t n, size_t at, cudaMemcpyKind,
                                      cudaStream_t) {
  const cudaError_t e = result("copy");
  if (e == cudaSuccess) memcpy(to, (const char*)symbol + at, n);
  return e;
}
cudaError_t cudaMemcpyToSymbolAsync(const void* symbol, const void* from, size_t n, size_t at,
                                    cudaMemcpyKind, cudaStream_t) {
  const cudaError_t e = result("copy");
  if (e == cudaSuccess) memcpy((char*)symbol + at, from, n);
  return e;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) {
  const cudaError_t e = result("sync");
  if (e == cudaSuccess && !poke_name.empty() && poke_after-- == 0) {
    *variable(poke_name) |= poke_value;
    poke_name.clear();
  }
  return e;
}
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return result("device");
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return result("attribute");
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  a->numRegs = 168;
  return result("function");
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return result("function"); }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = (void*)encoder;
  if (q) *q = cudaDriverEntryPointSuccess;
  return result("entry");
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
}
