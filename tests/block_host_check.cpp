// Host-side check of the C-ABI layer of the microscaled 4-bit linear, of layer
// norm and of the optimizer step, built with AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_block_abi_cpu.py. It runs only where
// no HIP device is visible: every call then ends in argument validation or in the
// device check, so the fake addresses are never dereferenced.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <vector>

#include "convrot.h"

namespace {

uint64_t g_state = 0x9E3779B97F4A7C15ull;
uint64_t next_u64() {   // SplitMix64
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
template <typename T, size_t N>
T pick(const T (&a)[N]) { return a[next_u64() % N]; }

void* const A = reinterpret_cast<void*>(0x100000);
void* const PTRS[] = {nullptr, A, A, A, A, A, A, A, A, reinterpret_cast<void*>(0x100004), reinterpret_cast<void*>(0x100002)};
const int64_t DIMS[] = {INT64_MIN, -1, 0, 1, 8, 17, 32, 64, 96, 128, 256, 1024, 4096, 16384, 16392, 32768, 32800, (int64_t)1 << 26,
                        (int64_t)1 << 31, (int64_t)1 << 40, INT64_MAX};
const int INTS[] = {INT32_MIN, -1, 0, 1, 2, 3, 8, 16, 32, 64, 256, 1024, 4096, 4097, 65536, 65537, INT32_MAX};
const size_t WSB[] = {0, 16, (size_t)1 << 20, (size_t)1 << 45, ~(size_t)0};
const double REALS[] = {-1.0, 0.0, 1e-8, 0.5, 0.9, 0.999, 1.0, 1e40, INFINITY, -INFINITY, NAN};

void* ptr() { return pick(PTRS); }
float* fptr() { return static_cast<float*>(pick(PTRS)); }
const int32_t* iptr() { return static_cast<const int32_t*>(pick(PTRS)); }
cr_out out() { return (cr_out)(next_u64() % 5); }

}  // namespace

int main() {
  if (convrot_device_check() != CR_ERR_NO_DEVICE) {
    std::printf("skipped: a HIP device is visible\n");
    return 0;
  }
  int fail = 0, reached = 0;
  std::vector<cr_adamw_tensor> list(70000);
  for (int r = 0; r < 400000; ++r) {
    const int64_t M = pick(DIMS), N = pick(DIMS), K = pick(DIMS);
    const int64_t lk = (next_u64() & 3) ? K : pick(DIMS), ln = (next_u64() & 3) ? N : pick(DIMS);
    const int S = (next_u64() & 1) ? 1 : pick(INTS);
    (void)convrot_layer_norm_backward_workspace_size(M, K, S);
    const int have = (int)(next_u64() % 4);
    for (int i = 0; i < have; ++i)
      list[(size_t)i] = cr_adamw_tensor{ptr(), ptr(), ptr(), ptr(), fptr(), fptr(), ptr(), pick(DIMS)};
    const bool easy = next_u64() & 1;
    const double beta = easy ? 0.9 : pick(REALS), real = easy ? 1e-3 : pick(REALS);
    const int bits = (next_u64() & 1) ? 32 : (next_u64() & 1) ? 8 : pick(INTS);
    const cr_status s[] = {
        mxfp4_quantize(ptr(), lk, M, K, pick(INTS), ptr(), ptr(), nullptr),
        mxfp4_dequantize(ptr(), ptr(), M, K, pick(INTS), ptr(), out(), lk, nullptr),
        mxfp4_gemm(ptr(), ptr(), ptr(), ptr(), ptr(), ptr(), out(), ln, M, N, K, nullptr),
        convrot_layer_norm_forward(ptr(), out(), lk, ptr(), lk, ptr(), ln, out(), (int)(next_u64() % 3), iptr(), S, real, ptr(), out(), lk,
                                   fptr(), fptr(), M, K, nullptr),
        convrot_layer_norm_backward(ptr(), out(), lk, ptr(), out(), lk, fptr(), fptr(), ptr(), ln, out(), (int)(next_u64() % 3), iptr(),
                                    S, ptr(), lk, ptr(), out(), lk, fptr(), fptr(), (int)(next_u64() & 1), M, K, ptr(), pick(WSB),
                                    nullptr),
        convrot_adamw_step(have ? list.data() : nullptr, have, out(), bits, real, beta, beta, real, real,
                           easy ? 1 : pick(DIMS), fptr(), (uint32_t)next_u64(), nullptr),
        convrot_adamw_moments(have ? list.data() : nullptr, have, fptr(), fptr(), nullptr)};
    for (cr_status v : s) {
      if ((int)v < 1 || (int)v > 7) {
        std::printf("FAIL status %d\n", (int)v);
        fail = 1;
      }
      reached += v == CR_ERR_NO_DEVICE;
    }
  }
  // the longest lists, with empty entries among them
  for (size_t i = 0; i < list.size(); ++i)
    list[i] = i % 3 ? cr_adamw_tensor{A, A, A, A, static_cast<float*>(A), static_cast<float*>(A), A, (int64_t)i} : cr_adamw_tensor{};
  for (int count : {1, 48, 49, 65536, 65537, INT32_MAX, -1}) {
    const cr_status v = convrot_adamw_step(list.data(), count, CR_OUT_F32, 8, 1e-3, 0.9, 0.999, 1e-8,
                                           0.01, 1, nullptr, 1, nullptr);
    if (v != (count >= 1 && count <= 65536 ? CR_ERR_NO_DEVICE : CR_ERR_UNSUPPORTED_SHAPE)) {
      std::printf("FAIL count %d status %d\n", count, (int)v);
      fail = 1;
    }
  }
  cr_counters c;
  convrot_get_counters(&c);
  for (uint64_t l : c.launches)
    if (l != 0) fail = 1;
  std::printf("%s: %d calls reached the device check\n", fail || !reached ? "FAILED" : "all ok", reached);
  return fail || !reached;
}
