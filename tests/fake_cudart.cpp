// A stand-in for the CUDA runtime that launches nothing: the host code of libspecverify.so runs against it on a machine
// without a device, and every launch is written down (kernel name, grid, block, thread that made it).
#include <chrono>
#include <cstddef>
#include <cstdio>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

struct Dim {
  unsigned x, y, z;
};
struct Config {   // the leading members of cudaLaunchConfig_t
  Dim grid, block;
  size_t smem;
  void* stream;
};

namespace {
std::mutex mu;
std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
struct Launch {
  std::string kernel;
  Dim grid, block;
  size_t thread;
};
std::vector<Launch>& launches() {
  static std::vector<Launch> v;
  return v;
}
int delay_ms = 0;
thread_local bool bound = false;   // a context is current on this thread
thread_local Config pushed;

int launch(const void* fn, Dim grid, Dim block) {
  {
    std::lock_guard<std::mutex> lk(mu);
    bound = true;
    launches().push_back({names()[fn], grid, block, std::hash<std::thread::id>()(std::this_thread::get_id())});
  }
  if (delay_ms) std::this_thread::sleep_for(std::chrono::milliseconds(delay_ms));
  return 0;
}
// cuTensorMapEncodeTiled: every cache can be described, by a thread that has a context (else CUDA_ERROR_INVALID_CONTEXT)
int encode(...) { return bound ? 0 : 201; }
}  // namespace

extern "C" {
void fake_delay(int ms) { delay_ms = ms; }
void fake_clear() {
  std::lock_guard<std::mutex> lk(mu);
  launches().clear();
}
int fake_count() {
  std::lock_guard<std::mutex> lk(mu);
  return static_cast<int>(launches().size());
}
void fake_get(int i, char* name, int room, unsigned* grid_block, size_t* thread) {
  std::lock_guard<std::mutex> lk(mu);
  const Launch& l = launches()[i];
  std::snprintf(name, room, "%s", l.kernel.c_str());
  std::memcpy(grid_block, &l.grid, sizeof(Dim));
  std::memcpy(grid_block + 3, &l.block, sizeof(Dim));
  *thread = l.thread;
}

void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* device, int, void*, void*, void*, void*, int*) {
  std::lock_guard<std::mutex> lk(mu);
  names()[host] = device;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
int __cudaGetKernel(const void** kernel, const void* host) {
  *kernel = host;
  return 0;
}
unsigned __cudaPushCallConfiguration(Dim grid, Dim block, size_t smem, void* stream) {
  pushed = {grid, block, smem, stream};
  return 0;
}
int __cudaPopCallConfiguration(Dim* grid, Dim* block, size_t* smem, void* stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *smem = pushed.smem;
  *static_cast<void**>(stream) = pushed.stream;
  return 0;
}
int __cudaLaunchKernel(const void* kernel, Dim grid, Dim block, void**, size_t, void*) { return launch(kernel, grid, block); }
int cudaLaunchKernel(const void* fn, Dim grid, Dim block, void**, size_t, void*) { return launch(fn, grid, block); }
int cudaLaunchKernelExC(const Config* c, const void* fn, void**) { return launch(fn, c->grid, c->block); }
int cudaDeviceGetAttribute(int* value, int, int) {
  *value = 152;
  return 0;
}
int cudaEventRecord(void*, void*) { return 0; }
int cudaFuncSetAttribute(const void*, int, int) { return 0; }
int cudaGetDevice(int* device) {
  *device = 0;
  return 0;
}
int cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long, int* found) {
  *fn = reinterpret_cast<void*>(&encode);
  *found = 0;
  return 0;
}
int cudaGetLastError() { return 0; }
int cudaGetSymbolAddress(void** at, const void*) {
  *at = nullptr;
  return 0;
}
int cudaMemcpyAsync(void*, const void*, size_t, int, void*) { return 0; }
int cudaMemsetAsync(void*, int, size_t, void*) { return 0; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, const void*, int, size_t) {
  *n = 2;
  return 0;
}
int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = 2;
  return 0;
}
int cudaOccupancyMaxActiveClusters(int* n, const void*, const void*) {
  *n = 8;
  return 0;
}
int cudaSetDevice(int) {
  bound = true;
  return 0;
}
int cudaStreamSynchronize(void*) { return 0; }
}
