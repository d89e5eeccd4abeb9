// The launches that attention's entry points make, without a GPU: this program has
// the runtime's launch functions, which the library (argv[1]) then finds here instead
// of the runtime's, and prints name, grid and block of each launch in place of making
// it, then "rc <status>".  No pointer that it passes is followed on the host.
//
//   decode  H_q H_kv d dtype packed N T max_len
//   bwd     H_q H_kv d dtype N T_q T_k
#include <dlfcn.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

#include "gdn.h"

struct Dim {
  uint32_t x, y, z;
};
static std::map<const void*, std::string>& names() {
  static std::map<const void*, std::string> m;
  return m;
}
static Dim g_grid, g_block;

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* module = nullptr;
  return &module;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*, void*, void*, void*, int*) {
  names()[host] = device;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
int __hipPushCallConfiguration(Dim grid, Dim block, size_t, void*) {
  g_grid = grid;
  g_block = block;
  return 0;
}
int __hipPopCallConfiguration(Dim* grid, Dim* block, size_t* shared, void** stream) {
  *grid = g_grid;
  *block = g_block;
  *shared = 0;
  *stream = nullptr;
  return 0;
}
int hipLaunchKernel(const void* f, Dim grid, Dim block, void**, size_t, void*) {
  std::printf("%s %u %u %u %u\n", names()[f].c_str(), grid.x, grid.y, grid.z, block.x * block.y * block.z);
  return 0;
}
int hipGetLastError() { return 0; }
}

int main(int argc, char** argv) {
  if (argc < 9) return 2;
  void* lib = dlopen(argv[1], RTLD_NOW);
  if (!lib) {
    std::fprintf(stderr, "%s\n", dlerror());
    return 3;
  }
  auto arg = [&](int i) { return std::atoll(argv[i]); };
  void* p = reinterpret_cast<void*>(4096);
  const int32_t* pi = static_cast<int32_t*>(p);
  float* pf = static_cast<float*>(p);
  const gdn_attn_shape_t s{static_cast<int32_t>(arg(3)), static_cast<int32_t>(arg(4)), static_cast<int32_t>(arg(5)),
                           static_cast<int32_t>(arg(6)), 0.125f};
  int rc = 4;
  if (!std::strcmp(argv[2], "decode") && argc == 11) {
    const bool packed = arg(7) != 0;
    const int32_t n = static_cast<int32_t>(arg(8));
    const int64_t T = arg(9), max_len = arg(10);
    const gdn_kv_cache_t c{p, p, pf, pf, 1 << 20, 1024};
    const auto call = reinterpret_cast<decltype(&gdn_attn_decode)>(dlsym(lib, "gdn_attn_decode"));
    const auto need = reinterpret_cast<decltype(&gdn_attn_decode_workspace_bytes)>(dlsym(lib, "gdn_attn_decode_workspace_bytes"));
    rc = call(&s, n, packed ? pi : nullptr, T, p, 0, &c, pi, 1 << 16, pi, max_len, p, 0, pf, p, need(&s, n, T, max_len), nullptr);
  } else if (!std::strcmp(argv[2], "bwd") && argc == 10) {
    const int32_t n = static_cast<int32_t>(arg(7));
    const int64_t Tq = arg(8), Tk = arg(9);
    const auto call = reinterpret_cast<decltype(&gdn_attn_bwd)>(dlsym(lib, "gdn_attn_bwd"));
    const auto need = reinterpret_cast<decltype(&gdn_attn_workspace_bytes)>(dlsym(lib, "gdn_attn_workspace_bytes"));
    rc = call(&s, n, pi, pi, Tq, Tk, p, 0, p, 0, p, 0, p, 0, pf, p, 0, p, 0, p, 0, p, 0, p, need(&s, Tq, Tk), nullptr);
  }
  std::printf("rc %d\n", rc);
  return 0;
}
