// Argument fuzzer for the host layer of the operators between token ids and the expert
// layer: random and extreme arguments, with addresses that must not be followed.  Meant
// for a machine without a GPU, where a call that passes the checks ends in a failed launch.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <random>

#include "nsg.h"

int main(int argc, char **argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 1000;
  std::mt19937_64 rng(54321);
  const int64_t sizes[] = {0, 1, 2, 7, 8, 63, 64, 65, 128, 1000, 1024, 1025, 4096, 65536, 65537, 1 << 20, (1 << 20) + 1, 1 << 25,
                           (1 << 25) + 1, 1ll << 31, (1ll << 31) + 1, 1ll << 40, INT64_MAX, -1, INT64_MIN};
  auto size = [&]() -> int64_t { return rng() % 3 ? (int64_t)(rng() % 300) : sizes[rng() % (sizeof sizes / sizeof *sizes)]; };
  auto code = [&]() -> int32_t { return rng() % 8 ? (int32_t)(rng() % 3) : (int32_t)rng(); };
  auto flag = [&]() -> int32_t { return rng() % 8 ? (int32_t)(rng() % 2) : (int32_t)rng(); };
  auto bits = [&]() -> int32_t { return rng() % 8 ? (rng() % 2 ? 64 : 32) : (int32_t)rng(); };
  auto real = [&]() -> float {
    const float v[] = {1.f, 0.f, 1e-5f, -1.f, 1e38f, std::numeric_limits<float>::infinity(), std::numeric_limits<float>::quiet_NaN()};
    return v[rng() % 3 ? 0 : rng() % 7];
  };
  auto ptr = [&]() -> void * {
    const int k = rng() % 10;
    return k == 0 ? nullptr : reinterpret_cast<void *>((uintptr_t)(0x10000 + (k == 1 ? rng() % 64 : 16 * (rng() % 64))));
  };
  long ok = 0, refused = 0, launched = 0;
  auto count = [&](nsg_status_t s) { (s == NSG_OK ? ok : s == NSG_ERR_HIP ? launched : refused)++; };
  for (int i = 0; i < n; ++i) {
    size_t bytes = 0;
    const int64_t T = size(), C = size(), V = size(), E = size(), k = rng() % 2 ? 1 + (int64_t)(rng() % 8) : size();
    auto ld = [&](int64_t c) { return rng() % 4 ? c : size(); };
    const size_t room = rng() % 2 ? (size_t)-1 : (size_t)size();
    count(nsg_embedding(ptr(), bits(), T, ptr(), code(), V, C, ld(C), real(), ptr(), nullptr));
    count(nsg_embedding_backward_workspace_size(T, V, C, rng() % 8 ? &bytes : nullptr));
    count(nsg_embedding_backward(ptr(), code(), T, C, ld(C), ptr(), bits(), V, real(), ptr(), code(), flag(), ptr(), room, nullptr));
    count(nsg_layer_norm(ptr(), code(), T, C, ld(C), ptr(), ptr(), code(), real(), ptr(), (float *)ptr(), nullptr));
    count(nsg_layer_norm_backward_workspace_size(T, C, rng() % 8 ? &bytes : nullptr));
    count(nsg_layer_norm_backward(ptr(), ld(C), ptr(), ld(C), code(), T, C, (float *)ptr(), ptr(), code(), ptr(), ptr(), ptr(), ptr(),
                                  room, nullptr));
    count(nsg_expert_route_workspace_size(T, E, rng() % 8 ? &bytes : nullptr));
    const bool b = rng() % 2;
    count(nsg_expert_route(ptr(), code(), T, E, ld(E), k, flag(), (float *)ptr(), (uint8_t *)ptr(), flag(), real(), (int32_t *)ptr(),
                           (float *)ptr(), b ? (int32_t *)ptr() : nullptr, b ? (float *)ptr() : nullptr, b ? (float *)ptr() : nullptr,
                           ptr(), room, nullptr));
    count(nsg_expert_route_backward(ptr(), code(), T, E, ld(E), k, flag(), flag(), real(), (int32_t *)ptr(), (float *)ptr(),
                                    (int32_t *)ptr(), real(), (float *)ptr(), ptr(), nullptr));
  }
  std::printf("ok %d iterations: %ld accepted, %ld refused, %ld up to the launch\n", n, ok, refused, launched);
  return refused > 0 && ok > 0 && launched > 0 ? 0 : 1;
}
