// What libkda.so hands to the HIP runtime, on the CPU: this program links the
// library and puts its own functions in place of the runtime's, so that every
// launch of a call is looked at and none is made.  The addresses are made up
// and never dereferenced.
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>
#include <string>

#include "kda_linear.h"
#include "kda_linear_internal.h"

static int failures = 0, launches = 0;
#define EXPECT(x)                                          \
  do {                                                     \
    if (!(x)) {                                            \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #x); \
      ++failures;                                          \
    }                                                      \
  } while (0)

static std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> m;
  return m;
}
static struct {
  dim3 grid, block;
  size_t shared;
  hipStream_t stream;
} config;

static void check_walk(const kda::LinearWalkArgs& w) {
  // a constant decay is read before the number of tokens is looked at
  EXPECT(!w.decay_per_head || w.log_decay);
}

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
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t shared, hipStream_t) {
  ++launches;
  const std::string& name = kernels()[f];
  EXPECT(!name.empty() && grid.x > 0 && grid.y == 1 && grid.z == 1 && block.y == 1 && block.z == 1);
  EXPECT(block.x > 0 && block.x <= 1024 && shared <= 160 * 1024);
  if ((uint64_t)grid.x * block.x > UINT32_MAX) {
    std::fprintf(stderr, "%s: %u blocks of %u threads\n", name.c_str(), grid.x, block.x);
    ++failures;
  }
  if (name.find("linear_walk_kernel") != std::string::npos || name.find("linear_states_kernel") != std::string::npos)
    check_walk(*static_cast<const kda::LinearWalkArgs*>(args[0]));
  if (name.find("linear_grad_kernel") != std::string::npos) {
    const kda::LinearGradArgs& g = *static_cast<const kda::LinearGradArgs*>(args[0]);
    check_walk(g.dq);
    check_walk(g.dk);
    check_walk(g.dv);
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

// an address space of its own for every tensor
template <typename T = void>
static T* P(int i) {
  return reinterpret_cast<T*>(0x100000000000ull + (uint64_t)i * 0x20000000000ull);
}

struct Sizes {
  int n;
  int64_t t;
  int h, hq, per_head, segment;
};
static size_t forward_bytes(const Sizes& z) {
  return kda_linear_chunk_fwd_workspace_bytes(z.n, z.t, z.h, z.hq, 128, 128, KDA_DTYPE_BF16, z.segment);
}
static int forward(const Sizes& z, const float* log_decay) {
  return kda_linear_chunk_fwd(P(0), P(1), P(2), log_decay, nullptr, z.n > 1 ? P<int32_t>(20) : nullptr, z.n, z.t, z.h,
                              z.hq, z.per_head, 128, 128, KDA_DTYPE_BF16, z.segment, P(4), P<float>(5), P(30),
                              forward_bytes(z), nullptr);
}
static int backward(const Sizes& z, const float* log_decay) {
  const size_t bytes = kda_linear_chunk_bwd_workspace_bytes(z.n, z.t, z.h, z.hq, z.per_head, 1, 0, 128, 128,
                                                            KDA_DTYPE_BF16, z.segment);
  return kda_linear_chunk_bwd(P(0), P(1), P(2), log_decay, nullptr, z.n > 1 ? P<int32_t>(20) : nullptr, P(6), nullptr,
                              z.n, z.t, z.h, z.hq, z.per_head, 128, 128, KDA_DTYPE_BF16, z.segment, P(8), P(9), P(10),
                              P<float>(11), nullptr, P(30), bytes, nullptr);
}

// Calls without tokens, which need no tensor of them: log_decay may be NULL.
static void no_tokens() {
  for (int n : {1, 3})
    for (int h : {2, 96, 300})
      for (int per_head : {0, 1})
        for (int segment : {-1, 0, 64}) {
          const Sizes z = {n, 0, h, h / 2, per_head, segment};
          EXPECT(forward(z, nullptr) == KDA_OK);
          EXPECT(backward(z, nullptr) == KDA_OK);
        }
}

// The last launch of the backward pass has a workgroup for each stretch of the
// decays' gradient and up to 2^20 for the sums of dq and as many for dk over
// shared heads; both at their limit, which the header gives as 14 * 2^20 for
// the former: tokens * heads / 1024 (/ 256) + 2 * sequences * heads.
static void most_stretches() {
  const Sizes at_limit[] = {{458240, 1 << 20, 16, 8, 0, -1}, {456704, 1 << 20, 16, 8, 1, -1}, {458240, 1 << 20, 16, 16, 0, -1}};
  for (const Sizes& z : at_limit) {
    EXPECT(z.t * z.h / (z.per_head ? 256 : 1024) + 2ll * z.n * z.h == 14ll << 20);
    EXPECT(backward(z, P<float>(3)) == KDA_OK);
    Sizes over = z;
    over.n += 1;
    EXPECT(backward(over, P<float>(3)) == KDA_ERR_INVALID_ARG);
  }
}

// Sizes from one token to the largest, every schedule.
static void sizes() {
  for (int n : {1, 2, 9, 1000, 400000})
    for (int h : {1, 3, 16, 48, 90, 96, 300, 65535})
      for (int64_t t : {1ll, 63ll, 4927ll, 131072ll, 3000000ll, 2147483647ll})
        for (int segment : {-1, 0, 64, 64 * 1021})
          for (int hq : {1, h})
            for (int per_head : {0, 1}) {
              const Sizes z = {n, t, h, hq, per_head, segment};
              if ((double)t * h > 1e9 || forward_bytes(z) >= 1ull << 40) continue;  // (2 TiB between the tensors)
              const int f = forward(z, P<float>(3)), b = backward(z, P<float>(3));
              EXPECT(f == KDA_OK || f == KDA_ERR_INVALID_ARG);
              EXPECT(b == KDA_OK || b == KDA_ERR_INVALID_ARG);
            }
}

int main(int argc, char** argv) {
  const std::string what = argc > 1 ? argv[1] : "";
  if (what == "no_tokens") no_tokens();
  else if (what == "most_stretches") most_stretches();
  else if (what == "sizes") sizes();
  else EXPECT(!"a known check");
  EXPECT(launches > 0);
  if (failures == 0) std::printf("%d launches checked\n", launches);
  return failures != 0;
}
