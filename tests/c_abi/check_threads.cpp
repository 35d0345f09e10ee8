// Precondition checks (KDA_DEBUG_CHECKS) of two threads at once, on the CPU: this
// program links libkda.so and puts its own functions in place of the HIP runtime's.
// They act out the checks' word in device memory: a launch that clears it does, a
// check launched by the thread whose inputs are bad sets a bit, a copy reads it.  The
// addresses of the calls are made up and never dereferenced.
#include <hip/hip_runtime_api.h>

#include <atomic>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <thread>

#include "kda.h"
#include "kda_delta.h"
#include "kda_linear.h"

static std::atomic<uint32_t> word{0};
static std::atomic<int> wrong{0}, checks{0};
static thread_local bool bad = false;

static std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> m;
  return m;
}
static thread_local struct {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} config;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*, int*) {
  kernels()[host] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream) {
  config = {grid, block, shared, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shared, hipStream_t* stream) {
  *grid = config.grid;
  *block = config.block;
  *shared = config.shared;
  *stream = config.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void**, size_t, hipStream_t) {
  const std::string& name = kernels().at(f);
  auto is = [&](const char* what) { return name.find(what) != std::string::npos; };
  if (is("flags_clear_kernel")) {
    word = 0;
  } else if (is("check_kernel") || is("check_rows_kernel")) {
    ++checks;
    if (bad) word |= 1;
  }
  std::this_thread::yield();
  return hipSuccess;
}
hipError_t hipMemsetAsync(void*, int, size_t, hipStream_t) {
  word = 0;
  std::this_thread::yield();
  return hipSuccess;
}
hipError_t hipGetSymbolAddress(void** p, const void*) {
  *p = &word;
  return hipSuccess;
}
hipError_t hipMemcpyAsync(void* to, const void*, size_t bytes, hipMemcpyKind, hipStream_t) {
  std::this_thread::yield();
  const uint32_t now = word;
  std::memcpy(to, &now, bytes);
  return hipSuccess;
}
hipError_t hipStreamSynchronize(hipStream_t) {
  std::this_thread::yield();
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
  *v = 256;
  return hipSuccess;
}
}

template <typename T = void>
static T* P(int i) {
  return reinterpret_cast<T*>(0x100000000000ull + (uint64_t)i * 0x20000000000ull);
}

static void calls(int which, bool is_bad) {
  bad = is_bad;
  for (int i = 0; i < 5000; ++i) {
    kda_status s;
    if (which == 0)
      s = kda_decode_step(P<float>(0), P(1), P(2), P(3), P<float>(4), P<float>(5), 1, 2, 128, 128, KDA_DTYPE_BF16, P(6),
                          nullptr);
    else if (which == 1)
      s = kda_linear_decode_step(P<float>(0), P(1), P(2), P(3), P<float>(4), 1, 2, 2, 0, 128, 128, KDA_DTYPE_BF16, P(6),
                                 nullptr);
    else
      s = kda_delta_decode_step(P<float>(0), P(1), P(2), P(3), P<float>(4), P<float>(5), 1, 2, 2, 128, 128, KDA_DTYPE_BF16,
                                P(6), nullptr);
    if (s != (is_bad ? KDA_ERR_PRECONDITION : KDA_OK) || kda_last_precondition_flags() != (is_bad ? 1u : 0u)) ++wrong;
  }
}

int main(int argc, char** argv) {
  setenv("KDA_DEBUG_CHECKS", "1", 1);
  const int which = argc > 1 ? std::atoi(argv[1]) : 0;
  std::thread a(calls, which, true), b(calls, which, false);
  a.join();
  b.join();
  std::printf("%d checks, %d wrong answers\n", (int)checks, (int)wrong);
  return wrong != 0 || checks < 10000;
}
