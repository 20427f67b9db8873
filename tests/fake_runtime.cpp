// Runs the library's entry points against a fake of the CUDA runtime calls on
// a launch's path, and prints which kernels they launch (test_launch_choice_cpu.py).
// The definitions here come before the runtime library's when symbols are
// looked up, so no driver and no GPU is needed and nothing is executed.
//
// Input, a command a line:
//   device D            makes D the current device
//   fail N              the next N cudaFuncSetAttribute calls fail
//   attention DT GROUP HKV DIM N MAX_Q N_REQ WIDTH PAGE WINDOW
//   plan N_REQ N_TOKENS
//   norm T D            (float32 throughout, RMS / RMS)
// Output, a line a command: {"status": .., "launches": [{"kernel": mangled name,
// "grid": .., "smem": .., "allowed": the dynamic shared memory that the current device lets that kernel have}]}
#include <cuda_runtime_api.h>
#include <dlfcn.h>

#include <cstdio>
#include <cstring>
#include <map>
#include <string>
#include <utility>

#include "gsi.h"

static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static int g_device = 0, g_fail = 0;
static std::map<std::pair<int, const void*>, int> g_allowed;
static std::string g_launches;
static const int kSms[2] = {152, 100};  // of device 0, and of any other

extern "C" {

void __cudaRegisterFunction(void** handle, const char* host, char* dev, const char* name, int limit, uint3* tid, uint3* bid,
                            dim3* bdim, dim3* gdim, int* wsize) {
  names()[host] = name;
  using Fn = void (*)(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*);
  reinterpret_cast<Fn>(dlsym(RTLD_NEXT, "__cudaRegisterFunction"))(handle, host, dev, name, limit, tid, bid, bdim, gdim, wsize);
}
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
  *v = a == cudaDevAttrMultiProcessorCount ? kSms[d != 0] : a == cudaDevAttrMaxSharedMemoryPerBlockOptin ? 232448 : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (g_fail > 0) {
    --g_fail;
    return cudaErrorInvalidValue;
  }
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_allowed[{g_device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  std::memset(a, 0, sizeof *a);
  a->numRegs = 168;
  return cudaSuccess;
}
static int fake_encode() { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&fake_encode);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  const auto it = g_allowed.find({g_device, f});
  char line[512];
  std::snprintf(line, sizeof line, "%s{\"kernel\": \"%s\", \"grid\": %u, \"smem\": %zu, \"allowed\": %d}",
                g_launches.empty() ? "" : ", ", names()[f].c_str(), c->gridDim.x, c->dynamicSmemBytes,
                it == g_allowed.end() ? 49152 : it->second);
  g_launches += line;
  return cudaSuccess;
}

}  // extern "C"

static void* const P = reinterpret_cast<void*>(0x100000);
static void* at(long long off) { return static_cast<char*>(P) + off; }

static int attention(int dt, long long group, long long hkv, long long dim, long long N, long long max_q, long long n_req,
                     long long width, long long page, long long window) {
  const gsi_cache_desc c{64, page, hkv, dim, gsi_dtype(dt), hkv * page * dim, page * dim, dim, P, P};
  const int32_t* ints = static_cast<const int32_t*>(P);
  return gsi_paged_attention(&c, P, group * hkv * dim, N, group * hkv, ints, ints, ints, width, n_req, max_q, 0.1f, 1, window,
                             P, P, size_t(1) << 40, nullptr);
}
static int plan(long long n_req, long long n_tokens) {
  int32_t* i = static_cast<int32_t*>(P);
  return gsi_paged_plan(i, i, n_req, i, 4, i, 4, i, 16, n_tokens, i, static_cast<int32_t*>(at(64)), static_cast<int64_t*>(P), i, i,
                        static_cast<int32_t*>(at(128)), i, nullptr);
}
static int norm(long long T, long long d) {
  const gsi_norm n{GSI_NORM_RMS, 1e-5f, static_cast<const float*>(P), nullptr};
  return gsi_norm_residual(P, GSI_F32, P, GSI_F32, T, d, 1.f, &n, nullptr, 0, nullptr, &n, P, P, GSI_F32, nullptr);
}

int main() {
  char line[512];
  while (std::fgets(line, sizeof line, stdin)) {
    long long v[10] = {};
    char op[32] = "";
    std::sscanf(line, "%31s %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", op, v, v + 1, v + 2, v + 3, v + 4, v + 5, v + 6,
                v + 7, v + 8, v + 9);
    g_launches.clear();
    int status = 0;
    if (!std::strcmp(op, "device"))
      g_device = int(v[0]);
    else if (!std::strcmp(op, "fail"))
      g_fail = int(v[0]);
    else if (!std::strcmp(op, "attention"))
      status = attention(int(v[0]), v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9]);
    else if (!std::strcmp(op, "plan"))
      status = plan(v[0], v[1]);
    else if (!std::strcmp(op, "norm"))
      status = norm(v[0], v[1]);
    else
      return 2;
    std::printf("{\"status\": %d, \"launches\": [%s]}\n", status, g_launches.c_str());
  }
  return 0;
}
