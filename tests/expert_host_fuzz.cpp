// Argument fuzzer for the host layer of the expert-layer entry points: random and
// extreme arguments, with addresses that must not be followed.  Meant for a machine
// without a GPU, where a call that passes the checks ends in a failed launch.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "nsg.h"

int main(int argc, char **argv) {
  const int n = argc > 1 ? std::atoi(argv[1]) : 1000;
  std::mt19937_64 rng(12345);
  const int64_t sizes[] = {0, 1, 2, 7, 8, 64, 127, 128, 129, 256, 1000, 4096, 65536, 65537, 1 << 20, 1 << 25, (1 << 25) + 1,
                           1ll << 31, 1ll << 40, INT64_MAX, -1, INT64_MIN};
  auto size = [&]() -> int64_t { return rng() % 3 ? (int64_t)(rng() % 300) : sizes[rng() % (sizeof sizes / sizeof *sizes)]; };
  auto code = [&]() -> int32_t { return rng() % 8 ? (int32_t)(rng() % 5) : (int32_t)rng(); };
  auto flag = [&]() -> int32_t { return rng() % 8 ? (int32_t)(rng() % 2) : (int32_t)rng(); };
  auto ptr = [&]() -> void * {
    const int k = rng() % 10;
    return k == 0 ? nullptr : reinterpret_cast<void *>((uintptr_t)(0x10000 + (k == 1 ? rng() % 64 : 16 * (rng() % 64))));
  };
  long ok = 0, refused = 0, launched = 0;
  auto count = [&](nsg_status_t s) { (s == NSG_OK ? ok : s == NSG_ERR_HIP ? launched : refused)++; };
  for (int i = 0; i < n; ++i) {
    size_t bytes = 0;
    int64_t cap = 0;
    count(nsg_expert_sort_workspace_size(size(), size(), size(), rng() % 8 ? &bytes : nullptr));
    count(nsg_fp8_columns(size(), size(), rng() % 8 ? &cap : nullptr));
    count(nsg_expert_sort(ptr(), rng() % 4 ? (rng() % 2 ? 64 : 32) : code(), size(), size(), size(), (int32_t *)ptr(), (int32_t *)ptr(),
                          (int32_t *)ptr(), ptr(), (size_t)size(), nullptr));
    count(nsg_expert_dispatch(ptr(), code(), size(), size(), size(), (int32_t *)ptr(), size(), (int32_t *)ptr(), size(), ptr(),
                              nullptr));
    count(nsg_expert_combine(ptr(), code(), size(), size(), size(), (int32_t *)ptr(), size(), size(), (float *)ptr(), ptr(),
                             nullptr));
    const int64_t T = size(), k = size(), C = size();
    const int64_t P = T > 0 && k > 0 && T < 1 << 25 && k < 1 << 25 ? T * k : size();
    count(nsg_expert_combine_backward(ptr(), C, ptr(), C, code(), P, C, (int32_t *)ptr(), size(), (int32_t *)ptr(), T, k,
                                      (float *)ptr(), ptr(), (float *)ptr(), nullptr));
    count(nsg_quantize_fp8(ptr(), code(), size(), size(), C, rng() % 2 ? C : size(), flag(), code(), ptr(), (float *)ptr(), ptr(),
                           (float *)ptr(), nullptr));
    count(nsg_quantize_fp8_columns(ptr(), code(), size(), C, C, (int32_t *)ptr(), size(), (int32_t *)ptr(), size(), code(), ptr(),
                                   (float *)ptr(), nullptr));
    const int64_t K = rng() % 2 ? 128 * (int64_t)(rng() % 100) : size();
    count(nsg_gemm_fp8_nt(code(), code(), code(), size(), size(), size(), K, ptr(), (float *)ptr(), flag(), ptr(),
                          (float *)ptr(), flag(), ptr(), nullptr));
    count(nsg_expert_gemm_fp8(code(), code(), code(), size(), size(), size(), size(), K, ptr(), (float *)ptr(), (int32_t *)ptr(),
                              ptr(), (float *)ptr(), flag(), (int32_t *)ptr(), ptr(), nullptr));
    count(nsg_expert_wgrad_fp8(code(), code(), code(), size(), size(), size(), size(), ptr(), (float *)ptr(), ptr(), (float *)ptr(),
                               (int32_t *)ptr(), ptr(), nullptr));
  }
  std::printf("ok %d iterations: %ld accepted, %ld refused, %ld up to the launch\n", n, ok, refused, launched);
  return refused > 0 && ok > 0 ? 0 : 1;
}
