// Host-side check of the C-ABI layer of the batched adapters and activation
// checkpoints, built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_adapter_abi_cpu.py. It runs only where no HIP device is visible:
// every call then ends in argument validation or in the device check, so the
// fake addresses are never dereferenced.
#include <cstdint>
#include <cstdio>

#include "convrot.h"

namespace {

uint64_t g_state = 0x2545F4914F6CDD1Dull;
uint64_t next_u64() {   // SplitMix64
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
template <typename T, size_t N>
T pick(const T (&a)[N]) { return a[next_u64() % N]; }

void* const A = reinterpret_cast<void*>(0x100000);
void* const PTRS[] = {nullptr, A, A, A, A, A, A, reinterpret_cast<void*>(0x100004)};
const int64_t DIMS[] = {INT64_MIN, -1, 0, 1, 8, 17, 64, 128, 256, 1024, 4096, 32768, 32776, 65536, (int64_t)1 << 26,
                        (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
const int INTS[] = {INT32_MIN, -1, 0, 1, 2, 3, 8, 16, 64, 128, 256, 1024, 4096, 4097, 65536, INT32_MAX};
const size_t WSB[] = {0, 16, (size_t)1 << 20, (size_t)1 << 45, ~(size_t)0};

void* ptr() { return pick(PTRS); }
float* fptr() { return static_cast<float*>(pick(PTRS)); }
const int32_t* iptr() { return static_cast<const int32_t*>(pick(PTRS)); }

}  // namespace

int main() {
  if (convrot_device_check() != CR_ERR_NO_DEVICE) {
    std::printf("skipped: a HIP device is visible\n");
    return 0;
  }
  int fail = 0, reached = 0;
  for (int r = 0; r < 400000; ++r) {
    const int64_t M = pick(DIMS), N = pick(DIMS), K = pick(DIMS);
    const int64_t lx = (next_u64() & 3) ? K : pick(DIMS), ly = (next_u64() & 3) ? N : pick(DIMS);
    const int R = pick(INTS), n = pick(INTS), S = pick(INTS);
    (void)convrot_lora_backward_workspace_size(M, N, K, R, n);
    const cr_status s[] = {
        convrot_lora_forward(ptr(), lx, ptr(), ptr(), R, n, iptr(), iptr(), S, fptr(), ptr(), ly, ptr(),
                             (cr_out)(next_u64() % 5), ly, fptr(), M, N, K, nullptr),
        convrot_lora_backward(ptr(), ly, fptr(), ptr(), lx, fptr(), (cr_gran)(next_u64() % 4), pick(INTS), ptr(), ptr(), R,
                              n, iptr(), iptr(), S, fptr(), ptr(), lx, ptr(), (cr_out)(next_u64() % 5), lx, fptr(), fptr(),
                              (int)(next_u64() & 1), M, N, K, ptr(), pick(WSB), nullptr),
        convrot_act_checkpoint(ptr(), lx, M, K, (cr_act)(next_u64() % 5), ptr(), lx, ptr(), fptr(), nullptr),
        convrot_act_backward(ptr(), lx, ptr(), fptr(), M, K, (cr_act)(next_u64() % 5), ptr(), lx, nullptr)};
    for (cr_status v : s) {
      if ((int)v < 1 || (int)v > 7) {
        std::printf("FAIL status %d\n", (int)v);
        fail = 1;
      }
      reached += v == CR_ERR_NO_DEVICE;
    }
  }
  cr_counters c;
  convrot_get_counters(&c);
  for (uint64_t l : c.launches)
    if (l != 0) fail = 1;
  std::printf("%s: %d calls reached the device check\n", fail || !reached ? "FAILED" : "all ok", reached);
  return fail || !reached;
}
