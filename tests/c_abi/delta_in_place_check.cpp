// In-place continuation of the gated delta rule (final_state == initial_state), on
// the CPU: this program links the library, puts its own functions in place of the
// HIP runtime's and looks at what every launch of a call is given.  The segments of
// a sequence are walked in any order, so no launch that walks a first segment apart
// from its last one may both read the initial state and write the final one.  The
// addresses are made up and never dereferenced.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <map>
#include <string>

#include "kda_delta.h"
#include "kda_delta_internal.h"

static int failures = 0, whole = 0, plain = 0, led = 0;
#define EXPECT(x)                                          \
  do {                                                     \
    if (!(x)) {                                            \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #x); \
      ++failures;                                          \
    }                                                      \
  } while (0)

template <typename T = void>
static T* P(int i) {
  return reinterpret_cast<T*>(0x100000000000ull + (uint64_t)i * 0x20000000000ull);
}
static float* const kState = P<float>(5);

static std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> m;
  return m;
}
static struct {
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
hipError_t hipLaunchKernel(const void* f, dim3, dim3, void** args, size_t, hipStream_t) {
  const std::string& name = kernels()[f];
  auto is = [&](const char* what) { return name.find(what) != std::string::npos; };
  if (is("delta_walk_kernel")) {
    const auto& a = *static_cast<const kda::DeltaWalkArgs*>(args[0]);
    EXPECT(a.fin == kState);
    if (!a.segmented) ++whole;
    else if (a.led) ++led;
    else ++plain;
    EXPECT((a.init == nullptr) == a.segmented);
  } else if (is("delta_pairs_kernel")) {
    // (led: it walks first segments only, and a workgroup that writes a final state has read that state itself)
    const auto& a = *static_cast<const kda::DeltaWalkArgs*>(args[0]);
    EXPECT(a.segmented && !a.all_pairs);
    EXPECT(a.init == (a.led ? kState : nullptr) && a.fin == (a.led ? kState : nullptr));
  } else if (is("delta_scan_kernel")) {
    const auto& a = *static_cast<const kda::DeltaScanArgs*>(args[0]);
    EXPECT(a.init == kState);
  } else {
    EXPECT(is("delta_prep_kernel"));
  }
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

static void call(int n, int64_t t, int h, kda_dtype dt, int seg) {
  const size_t bytes = kda_delta_chunk_fwd_workspace_bytes(n, t, h, h, 128, 128, dt, seg);
  EXPECT(kda_delta_chunk_fwd(P(0), P(1), P(2), P<float>(3), P<float>(12), kState, n > 1 ? P<int32_t>(20) : nullptr, n, t, h,
                             h, 128, 128, dt, seg, P(4), kState, P(30), bytes, nullptr) == KDA_OK);
}

int main() {
  for (kda_dtype dt : {KDA_DTYPE_F32, KDA_DTYPE_BF16})
    for (int n : {1, 2, 9, 300})
      for (int h : {1, 2, 8, 32, 96})
        for (int64_t t : {0ll, 1ll, 65ll, 1024ll, 8192ll, 131072ll})
          for (int seg : {-1, 0, 64, 1024}) call(n, t, h, dt, seg);
  // what a caller meets without asking for segments, in the form in which the first segments are not walked ahead
  plain = 0;
  call(1, 8192, 8, KDA_DTYPE_BF16, 0);
  call(1, 8192, 8, KDA_DTYPE_F32, 0);
  call(1, 1024, 2, KDA_DTYPE_BF16, 0);
  EXPECT(plain == 3);
  EXPECT(whole > 100 && led > 100);
  if (failures == 0) std::printf("in-place launches checked\n");
  return failures != 0;
}
